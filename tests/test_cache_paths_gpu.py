"""Ways through the bounded cache's kernels that need more sequences, longer caches or other calls at the same time."""
import math

import pytest
from test_cache_gpu import i32, kept_rows, nan_rows, random_cache, rnd, values64, weights_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sdpa(cuda_device):
    import memory_optimal_sdpa_b200 as m
    yield m
    assert m.get_last_device_error() == m.SDPA_OK


# ------------------------------------------------------------------------------------------ more than 32 sequences
LENGTHS = {
    "32": [7 * b % 90 for b in range(32)],
    "33": [0] * 32 + [90],
    "40, empty at the end": [11 * b % 91 for b in range(8)] + [0] * 31 + [64],
    "70": [13 * b % 91 for b in range(70)],
    "70, empty at both ends": [0] * 35 + [90, 1, 0, 64, 65] + [0] * 30,
    "100, equal": [33] * 100,
    "64, one long": [0] * 63 + [2000],
}


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 3, 3), (128, 8, 2), (64, 40, 2)])
@pytest.mark.parametrize("kind", list(LENGTHS))
def test_decode_of_many_sequences(sdpa, kind, d, Hq, Hkv, bits):
    """Each sequence gives what it gives alone, to the rounding of its sums in another order."""
    import torch
    lens = LENGTHS[kind]
    B, cap, G = len(lens), max(max(lens), 91), Hq // Hkv
    q = rnd((B, Hq, d), 1)
    acc = rnd((B, Hkv, cap), 2).float().abs()
    before = acc.clone()
    if bits == 4:
        c = random_cache(sdpa, B, Hkv, cap, d, lens, 3)
        k, v = values64(c.k_codes, c.k_scales), values64(c.v_codes, c.v_scales)
        O, L = sdpa.decode_kv4(q, c, i32(lens), acc=acc)
    else:
        kb, vb = nan_rows(rnd((B, Hkv, cap, d), 3), lens), nan_rows(rnd((B, Hkv, cap, d), 4), lens)
        k, v = kb.double(), vb.double()
        O, L = sdpa.decode_acc(q, kb, vb, i32(lens), acc)
    for b, n in enumerate(lens):
        assert torch.equal(acc[b, :, n:], before[b, :, n:])
        if n == 0:
            assert (O[b] == 0).all() and (L[b] == -math.inf).all()
            continue
        s = q[b].double().view(Hkv, G, d) @ k[b, :, :n].transpose(-1, -2) * d ** -0.5
        p = torch.softmax(s, -1)
        # scores of a few units, held in 32 bits with d / 16 + 8 units of 2^-23 |q| |k| scale < 2^6 each: below 2^-12
        rel = 2.0 ** -12
        want, size = (p @ v[b, :, :n]).view(Hq, d), (p @ v[b, :, :n].abs()).view(Hq, d)
        assert ((O[b].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 if bits == 4 else 2 * rel) * size).all(), b
        assert ((L[b].double() - torch.logsumexp(s, -1).view(-1)).abs() <= rel).all(), b
        assert ((acc[b, :, :n].double() - before[b, :, :n].double() - p.sum(1)).abs() <= 2 * rel * p.sum(1) + 2.0 ** -20).all(), b


# ------------------------------------------------------------------------------------------ weights beyond shared memory
@pytest.mark.parametrize("kind", ["plain", "ties", "special", "equal"])
@pytest.mark.parametrize("cap,n_out,n,budget,recent", [
    (49152, None, 49152, 20000, 100), (49153, None, 49153, 20000, 100), (49153, None, 49153, 49153, 0), (60001, None, 59999, 1025, 1024),
    (60001, 3000, 60001, 2999, 0), (60001, 60001, 30000, 30001, 64), (50000, None, 777, 40000, 40000), (49153, None, 0, 1, 1), (200001, 4096, 200001, 4096, 33)])
def test_evict_from_long_caches(sdpa, cap, n_out, n, budget, recent, kind):
    import torch
    d, H = 64, 2
    acc = nan_rows(weights_for(kind, (1, H, cap), 7), [n])
    k, v = nan_rows(rnd((1, H, cap, d), 1), [n]), nan_rows(rnd((1, H, cap, d), 2), [n])
    old = [t.clone() for t in (k, v, acc)]
    if n_out is None:
        k2, v2, a2, kw = k, v, acc, {}
    else:
        k2, v2 = (torch.full((1, H, n_out, d), 3.0, dtype=k.dtype, device="cuda") for _ in "kv")
        a2 = torch.full((1, H, n_out), 3.0, device="cuda")
        kw = dict(k_out=k2, v_out=v2, acc_out=a2)
    tails = [t.clone() for t in (k2, v2)]
    keep, new = sdpa.evict(k, v, acc, i32([n]), budget, recent=recent, **kw)
    bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    assert new.tolist() == [min(n, budget)]
    for h in range(H):
        rows = kept_rows(old[2][0, h].cpu(), n, budget, recent)
        m = len(rows)
        assert keep[0, h].tolist() == rows + [-1] * (budget - m)
        assert torch.equal(bits(a2[0, h, :m]), bits(old[2][0, h, rows])) and (a2[0, h, m:] == 0).all()
        for o, src, tail in ((k2, old[0], tails[0]), (v2, old[1], tails[1])):
            assert torch.equal(bits(o[0, h, :m]), bits(src[0, h, rows])) and torch.equal(bits(o[0, h, m:]), bits(tail[0, h, m:]))


# ------------------------------------------------------------------------------------------ lengths out of range
def fenced(like, fill):
    """A tensor of this shape between two others of it that hold `fill`, and the three as one."""
    import torch
    whole = torch.full((3, *like.shape), fill, dtype=like.dtype, device="cuda")
    whole[1] = like
    return whole[1], whole


@pytest.mark.parametrize("lens,n_new,true_lens,true_new", [
    ([6, 0], None, [6, 0], [2, 4]), ([9, 1], None, [8, 1], [0, 4]), ([-1, 0], None, [0, 0], [4, 4]), ([0, 2], [5, 1], [0, 2], [4, 1]),
    ([3, 0], [-1, 4], [3, 0], [0, 4]), ([8, 7], [4, 4], [8, 7], [0, 1]), ([2147483647, -2147483648], [4, 4], [8, 0], [0, 4])])
@pytest.mark.parametrize("d", [64, 128])
def test_append_stays_inside_the_cache(sdpa, d, lens, n_new, true_lens, true_new):
    """Lengths out of range do what the nearest ones in range do, and are reported; nothing else of the cache or beside it changes."""
    import torch
    cap = 8
    k, v = rnd((2, 3, 4, d), 1), rnd((2, 3, 4, d), 2)
    made = []
    for at, new in ((lens, n_new), (true_lens, true_new)):
        parts = [fenced(torch.full_like(t, 7), 9) for t in sdpa.kv4_cache(2, 3, cap, d)]
        reads = [fenced(torch.full_like(k, 7), 9) for _ in "kv"]
        sdpa.kv4_append(sdpa.Kv4Cache(*(p[0] for p in parts)), k, v, i32(at), n_new=None if new is None else i32(new), k_read=reads[0][0], v_read=reads[1][0])
        assert sdpa.get_last_device_error() == (sdpa.SDPA_OK if made else sdpa.SDPA_ERR_DEVICE_BAD_LENGTH)
        made.append([p[1] for p in parts + reads])
    for a, b in zip(*made):
        assert torch.equal(a, b) and (a[0] == 9).all() and (a[2] == 9).all()


@pytest.mark.parametrize("lens,true_lens", [([9, 1], [8, 1]), ([-1, 3], [0, 3]), ([2147483647, -2147483648], [8, 0])])
def test_reads_stay_inside_the_cache(sdpa, lens, true_lens):
    import torch
    d, cap, bad = 64, 8, sdpa.SDPA_ERR_DEVICE_BAD_LENGTH
    cache = random_cache(sdpa, 2, 3, cap, d, [cap, cap], 1)
    q, kb, vb = rnd((2, 6, d), 2), rnd((2, 3, cap, d), 3), rnd((2, 3, cap, d), 4)
    acc0 = rnd((2, 3, cap), 5).float().abs()

    def everything(at):
        n, out = i32(at), []

        def done(*tensors):
            assert sdpa.get_last_device_error() == (sdpa.SDPA_OK if at == true_lens else bad)
            out.extend(tensors)
        for call in (lambda a: sdpa.decode_kv4(q, cache, n, acc=a), lambda a: sdpa.decode_acc(q, kb, vb, n, a)):
            acc, whole = fenced(acc0, 9.0)
            done(*call(acc), whole)
        K, V = (fenced(torch.full((2, 3, cap, d), 7.0, device="cuda").to(torch.bfloat16), 9.0) for _ in "kv")
        sdpa.kv4_load(cache, n, k=K[0], v=V[0])
        done(K[1], V[1])
        k, v, acc = fenced(kb, 9.0), fenced(vb, 9.0), fenced(acc0, 9.0)
        done(*sdpa.evict(k[0], v[0], acc[0], n, 3, recent=1), k[1], v[1], acc[1])
        parts, acc = [fenced(t, 9) for t in cache], fenced(acc0, 9.0)
        done(*sdpa.kv4_evict(sdpa.Kv4Cache(*(p[0] for p in parts)), acc[0], n, 3), *(p[1] for p in parts), acc[1])
        return out
    for a, b in zip(everything(lens), everything(true_lens)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------ calls at the same time
def test_calls_beside_a_replayed_graph(sdpa):
    """A decode step replayed on one stream while other decodes, appends and evictions run on another: all give what they give alone."""
    import torch
    d, B, Hq, Hkv, cap = 128, 6, 16, 4, 1500
    q, kn, vn = rnd((B, Hq, d), 1), rnd((B, Hkv, 1, d), 2), rnd((B, Hkv, 1, d), 3)
    lens0 = [1000, 0, 37, 1400, 511, 900]

    def fresh(seed):
        c = random_cache(sdpa, B, Hkv, cap, d, [cap] * B, seed)
        return c, torch.zeros((B, Hkv, cap), device="cuda"), i32(lens0)

    def step(c, acc, lens):
        sdpa.kv4_append(c, kn, vn, lens)
        lens += 1
        return sdpa.decode_kv4(q, c, lens, acc=acc)

    def others(c, k, v, acc, n):
        O, L = sdpa.decode_acc(q, k, v, n, acc)
        keep, new = sdpa.kv4_evict(c, acc, n, 300, recent=20)
        return (O, L, keep, new, *sdpa.decode_kv4(q, c, new, acc=acc), sdpa.kv4_load(c, new, n_rows=300)[0])
    rounds = 25
    alone = fresh(5)
    steps = [[t.clone() for t in step(*alone)] for _ in range(rounds)]
    k, v, n = rnd((B, Hkv, cap, d), 7), rnd((B, Hkv, cap, d), 8), i32([900, 1500, 1, 0, 700, 333])
    want = [t.clone() for t in others(random_cache(sdpa, B, Hkv, cap, d, [cap] * B, 6), k, v, torch.zeros((B, Hkv, cap), device="cuda"), n)]

    state = fresh(5)
    warm = fresh(9)
    step(*warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*state)
    caches = [random_cache(sdpa, B, Hkv, cap, d, [cap] * B, 6) for _ in range(rounds)]
    sums = [torch.zeros((B, Hkv, cap), device="cuda") for _ in range(rounds)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    replays, beside = [], []
    for i in range(rounds):
        with torch.cuda.stream(side):
            graph.replay()
            replays.append([t.clone() for t in got])
        beside.append(others(caches[i], k, v, sums[i], n))
    torch.cuda.synchronize()
    for a, b in zip(replays, steps):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(state[1], alone[1]) and all(torch.equal(x, y) for x, y in zip(state[0], alone[0]))
    for r in beside:
        assert all(torch.equal(x, y) for x, y in zip(r, want))


# ------------------------------------------------------------------------------------------ prompts about the border of the two unit sizes
@pytest.mark.parametrize("B,Hq,Hkv,n_q,n_kv,d", [(4, 8, 8, 1300, 1300, 64), (4, 8, 8, 1100, 1300, 128), (4, 16, 8, 260, 1300, 64), (4, 8, 8, 140, 1300, 128),
                                                 (6, 8, 8, 128, 1024, 64), (5, 8, 8, 128, 1024, 64), (4, 8, 8, 1300, 700, 128), (9, 8, 8, 513, 513, 64)])
@pytest.mark.parametrize("causal", [False, True])
def test_prompt_weights(sdpa, B, Hq, Hkv, n_q, n_kv, d, causal):
    import torch
    q, k = rnd((B, Hq, n_q, d), 1), rnd((B, Hkv, n_kv, d), 2)
    G, want = Hq // Hkv, torch.zeros((B, Hkv, n_kv), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, Hq, n_q), device="cuda")
    seen = torch.arange(n_kv, device="cuda") <= torch.arange(n_q, device="cuda")[:, None] + (n_kv - n_q)
    for b in range(B):
        s = q[b].double() @ k[b].repeat_interleave(G, 0).double().transpose(-1, -2) * d ** -0.5
        if causal:
            s.masked_fill_(~seen, -math.inf)
        lse[b] = torch.logsumexp(s, -1).float()
        w = torch.exp(s - lse[b, ..., None].double()).nan_to_num(nan=0.0)  # queries that see no key
        want[b] = w.view(Hkv, G, n_q, n_kv).sum((1, 2))
    acc = sdpa.fwd_acc(q, k, lse, causal=causal)
    # scores of a few units, off by less than 2^-12; the sums by 2^-22 for each of their sqrt(n) steps
    rel = 2.0 ** -12 + 2.0 ** -22 * math.sqrt(n_q * G)
    assert ((acc.double() - want).abs() <= rel * want + n_q * G * 2.0 ** -126).all()
    assert torch.equal(acc, sdpa.fwd_acc(q, k, lse, causal=causal))
