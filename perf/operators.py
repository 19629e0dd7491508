"""Workloads of the bounded-cache operators: the 4-bit key/value cache and eviction by accumulated weight.

`run(state)` computes one pass of an operator, in plain torch operations where `own` is false and
through memory_optimal_sdpa_b200 where it is true.  The six operators:

  decode   attention of one query row per head over a 4-bit cache               decode_kv4
  acc      the same, or over a bf16 cache, adding each key's weight to `acc`    decode_kv4 / decode_acc
  append   new rows quantised into a 4-bit cache                                kv4_append
  load     the rows of a 4-bit cache as bf16                                    kv4_load
  prompt   each key's weight summed over the queries of a prompt                fwd_acc
  evict    the rows of largest accumulated weight and the most recent ones      evict / kv4_evict

A 4-bit cache row holds d channels in groups of 32.  A group has a scale s and a minimum m (bf16) and a
code c in 0 .. 15 for each channel, which stands for s c + m.  Byte 2 (r NG + g) + e of a row (NG = d / 32
groups; r in 0 .. 7, g in 0 .. NG - 1, e in 0 .. 1) holds channel 32 g + 4 r + 2 e in its low four bits
and the next channel in its high four.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one user's chat: a single sequence, a short cache; latency is what counts
        dict(name="decode_one", op="decode", batch=1, heads_q=32, heads_kv=8, d=128, cap=1024, lo=777, hi=777),
        # a full serving batch: 64 sequences of 1024 to 16384 tokens, 64 query heads over 8
        dict(name="decode_batch", op="decode", batch=64, heads_q=64, heads_kv=8, d=128, cap=16384, lo=1024, hi=16384),
        # 4-bit multi-head cache with weights kept for eviction; one slot of the batch is empty, odd capacity
        dict(name="acc_kv4_mha", op="acc", bits=4, batch=8, heads_q=16, heads_kv=16, d=64, cap=8191, lo=0, hi=8191),
        # long documents over a bf16 cache, weights kept for eviction
        dict(name="acc_bf16_long", op="acc", bits=16, batch=4, heads_q=32, heads_kv=8, d=128, cap=32768, lo=20001, hi=32768),
        # the decode step's own append: one token a sequence
        dict(name="append_token", op="append", batch=64, heads=8, d=128, cap=2048, lo=100, hi=1999, rows=1, rows_lo=1),
        # padded prompts of a batch written into the cache after prefill
        dict(name="append_prompt", op="append", batch=4, heads=8, d=128, cap=16384, lo=0, hi=777, rows=8192, rows_lo=5001),
        # the next turn of a short chat reads its cache for the prefill
        dict(name="load_turn", op="load", batch=1, heads=8, d=64, cap=2048, lo=1501, hi=1501),
        # the next turn after long documents
        dict(name="load_long", op="load", batch=4, heads=8, d=128, cap=16384, lo=9001, hi=16384),
        # every query of a prompt, causal: 32 query heads over 8, n = 8192
        dict(name="prompt_all", op="prompt", batch=1, heads_q=32, heads_kv=8, d=128, n_q=8192, n_kv=8192, causal=True),
        # the last 64 queries of long prompts as the window that decides what is kept
        dict(name="prompt_window", op="prompt", batch=4, heads_q=16, heads_kv=16, d=64, n_q=64, n_kv=16001, causal=True),
        # prompts cut to a quarter after prefill
        dict(name="evict_prompt", op="evict", bits=16, batch=16, heads=8, d=128, cap=8192, lo=4001, hi=8192, budget=2048, recent=256),
        # a 4-bit cache cut, then read back for the next turn; some sequences are shorter than the budget
        dict(name="evict_kv4", op="evict", bits=4, batch=2, heads=8, d=64, cap=2000, lo=400, hi=1999, budget=512, recent=33),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("decode", "acc", "append", "load", "prompt", "evict"))
    d = rng.choice((64, 128))
    if op in ("decode", "acc"):
        bits = 4 if op == "decode" else rng.choice((4, 16))
        heads_kv, group = _log(rng, 1, 16), rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 12, 16, 20))
        batch = _log(rng, 1, 32)
        most = (1 << 28) if bits == 4 else (1 << 26)
        cap = _log(rng, 16, max(32, min(65536, most // (batch * heads_kv * d))))
        hi = rng.randint(1, cap)
        case = dict(op=op, batch=batch, heads_q=heads_kv * group, heads_kv=heads_kv, d=d, cap=cap, lo=rng.randint(0, hi), hi=hi)
        return dict(case, bits=bits) if op == "acc" else case
    if op == "append":
        batch, heads = _log(rng, 1, 32), _log(rng, 1, 16)
        rows = _log(rng, 1, max(2, min(8192, (1 << 25) // (batch * heads * d))))
        hi = _log(rng, 1, 1024)
        return dict(op=op, batch=batch, heads=heads, d=d, cap=hi + rows + rng.randint(0, 100), lo=rng.randint(0, hi), hi=hi, rows=rows, rows_lo=rng.randint(0, rows))
    if op == "load":
        batch, heads = _log(rng, 1, 16), _log(rng, 1, 16)
        cap = _log(rng, 16, max(32, min(32768, (1 << 26) // (batch * heads * d))))
        hi = rng.randint(1, cap)
        return dict(op=op, batch=batch, heads=heads, d=d, cap=cap, lo=rng.randint(0, hi), hi=hi)
    if op == "prompt":
        heads_kv, group, batch = _log(rng, 1, 8), rng.choice((1, 1, 2, 3, 4, 5, 8)), _log(rng, 1, 4)
        most = (1 << 28) // (batch * heads_kv * group)
        n_kv = _log(rng, 1, min(16384, most))
        n_q = min(n_kv, _log(rng, 1, max(1, min(8192, most // n_kv))))
        return dict(op=op, batch=batch, heads_q=heads_kv * group, heads_kv=heads_kv, d=d, n_q=n_q, n_kv=n_kv, causal=rng.random() < 0.7)
    batch, heads = _log(rng, 1, 16), _log(rng, 1, 16)
    cap = _log(rng, 16, max(32, min(32768, (1 << 26) // (batch * heads * d))))
    budget, hi = rng.randint(1, cap), rng.randint(1, cap)
    return dict(op=op, bits=rng.choice((4, 16)), batch=batch, heads=heads, d=d, cap=cap, lo=rng.randint(0, hi), hi=hi, budget=budget, recent=rng.randint(0, min(budget, 300)))


# ------------------------------------------------------------------------------------------ inputs
def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly apart (hi alone for n = 1)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


class _Make:
    def __init__(self, seed):
        self.dev = torch.device("cuda", torch.cuda.current_device())
        self.gen = torch.Generator(device=self.dev)
        self.gen.manual_seed(seed)
        self.order = torch.Generator().manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=BF16):
        return (torch.randn(shape, generator=self.gen, device=self.dev, dtype=F32) * std).to(dtype)

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.gen, device=self.dev, dtype=F32)

    def shuffled(self, values):
        at = torch.randperm(len(values), generator=self.order)
        return torch.tensor(values, dtype=torch.int32)[at]

    def cache4(self, batch, heads, cap, d):
        """Codes, scales and minima as quantised normal rows have them, some groups with an offset of their own."""
        ng = d // 32
        codes = torch.empty((batch, heads, cap, d // 2), dtype=torch.uint8, device=self.dev)
        for b in range(batch):
            c = self.normal(2, heads, cap, d // 2, std=3.2, dtype=F32).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
            codes[b] = c[0] | (c[1] << 4)
        s = 0.2 + 0.25 * self.uniform(batch, heads, cap, ng)
        m = -s * (7.0 + self.uniform(batch, heads, cap, ng)) + 0.5 * self.normal(1, heads, 1, ng, dtype=F32)
        return codes, torch.stack((s, m), -1).to(BF16)

    def weights(self, batch, heads, cap):
        """Accumulated attention weights: a few keys hold most of them."""
        return (self.normal(batch, heads, cap, std=2.0, dtype=F32) - 3.0).exp_()


def _dims(case):
    return tuple(case[k] for k in ("batch", "heads_q" if "heads_q" in case else "heads", "d"))


def prepare(case, seed):
    make, op = _Make(seed), case["op"]
    B, H, d = _dims(case)
    st = {"case": case, "op": op}
    if op == "prompt":
        Hkv, n_q, n_kv = case["heads_kv"], case["n_q"], case["n_kv"]
        st["q"], st["k"] = make.normal(B, H, n_q, d), make.normal(B, Hkv, n_kv, d)
        st["acc"], st["acc_out"] = make.weights(B, Hkv, n_kv), torch.zeros((B, Hkv, n_kv), device=make.dev)
        # the log-sum-exps that the prefill of these queries gave
        lse = torch.empty((B, H, n_q), device=make.dev)
        for b in range(B):
            for h in range(H):
                for i in range(0, n_q, 2048):
                    s = st["q"][b, h, i:i + 2048].float() @ st["k"][b, h * Hkv // H].float().T / math.sqrt(d)
                    if case["causal"]:
                        at = torch.arange(i, i + s.shape[0], device=make.dev)[:, None] + (n_kv - n_q)
                        s.masked_fill_(torch.arange(n_kv, device=make.dev) > at, -math.inf)
                    lse[b, h, i:i + 2048] = torch.logsumexp(s, -1)
        st["lse"] = lse
        return st
    cap = case["cap"]
    lens = make.shuffled(_spread(case["lo"], case["hi"], B))
    st["lens"] = lens.to(make.dev)
    Hkv = case.get("heads_kv", H)
    ng = d // 32
    if op == "append":
        T = case["rows"]
        new = make.shuffled(_spread(case["rows_lo"], T, B))
        st["k"], st["v"] = make.normal(B, H, T, d), make.normal(B, H, T, d)
        st["k"] += make.normal(1, H, 1, d, std=0.7)  # keys have channels with an offset
        st["n_new"] = new.to(make.dev)
        for name in ("k", "v"):
            st[name + "_codes"] = torch.zeros((B, H, cap, d // 2), dtype=torch.uint8, device=make.dev)
            st[name + "_scales"] = torch.zeros((B, H, cap, ng, 2), dtype=BF16, device=make.dev)
            st[name + "_read"] = torch.zeros((B, H, T, d), dtype=BF16, device=make.dev)
        # sequence, row among the new ones and cache row of everything that is written
        b = torch.repeat_interleave(torch.arange(B), new.long())
        t = torch.cat([torch.arange(int(n)) for n in new])
        st["at"] = tuple(x.to(make.dev) for x in (b, t, lens.long()[b] + t))
        return st
    if op in ("decode", "acc"):
        st["q"] = make.normal(B, H, d, std=1.2)
    if op == "acc":
        st["acc"] = make.weights(B, Hkv, cap)
        st["acc_out"] = st["acc"].clone()
    if case.get("bits", 4) == 4:
        for name in ("k", "v"):
            st[name + "_codes"], st[name + "_scales"] = make.cache4(B, Hkv, cap, d)
    else:
        st["k"], st["v"] = make.normal(B, Hkv, cap, d), make.normal(B, Hkv, cap, d)
    if op == "load":
        n = case["hi"]
        st["k_out"], st["v_out"] = (torch.zeros((B, H, n, d), dtype=BF16, device=make.dev) for _ in range(2))
    if op == "evict":
        n = case["budget"]
        st["acc"] = make.weights(B, H, cap)
        st["acc_out"] = torch.zeros((B, H, n), device=make.dev)
        st["k_out"], st["v_out"] = (torch.zeros((B, H, n, d), dtype=BF16, device=make.dev) for _ in range(2))
        if case["bits"] == 4:
            for name in ("k", "v"):
                st[name + "_codes_out"] = torch.zeros((B, H, n, d // 2), dtype=torch.uint8, device=make.dev)
                st[name + "_scales_out"] = torch.zeros((B, H, n, ng, 2), dtype=BF16, device=make.dev)
    return st


# ------------------------------------------------------------------------------------------ plain forms
def _unpack(codes, scales):
    """Codes and scales of a 4-bit cache as the fp32 values they stand for."""
    ng = scales.shape[-2]
    c = codes.view(*codes.shape[:-1], 8, ng, 2)
    c = torch.stack((c & 15, c >> 4), -1).transpose(-4, -3).reshape(*codes.shape[:-1], ng, 32)
    s = scales.float()
    return (c.float() * s[..., :1] + s[..., 1:]).flatten(-2)


def _quantise(x):
    """Codes in 0 .. 15 (channel order), scales and minima of rows; in 64 bits, as codes next to a border need."""
    g = x.double().unflatten(-1, (-1, 32))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    want = (hi - lo) / 15
    s = want.to(BF16)
    s = torch.where(s.double() < want, (s.view(torch.int16) + 1).view(BF16), s)  # the next bf16 not below
    c = torch.where(s > 0, torch.round((g - lo) / s.double()), torch.zeros_like(g))
    return c, torch.cat((s, lo.to(BF16)), -1)


def _pack(c):
    """Codes [..., NG, 32] as the bytes of a cache row."""
    c = c.to(torch.uint8).unflatten(-1, (8, 2, 2)).transpose(-4, -3)
    return (c[..., 0] | (c[..., 1] << 4)).flatten(-3)


def _attend(q, k, v, lens):
    """o, lse and weights [B, Hkv, G, n] of one query row per head over fp32 keys and values."""
    B, Hkv, n, d = k.shape
    s = (q.float().view(B, Hkv, -1, d) @ k.transpose(-1, -2)) / math.sqrt(d)
    s.masked_fill_(torch.arange(n, device=k.device) >= lens[:, None, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(torch.finfo(F32).min)
    p = (s - m).exp_()
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, torch.ones_like(l))
    return (p @ v).view(B, -1, d).to(BF16), (m + l.log()).view(B, -1), p


def _written(lens, n):
    return (torch.arange(n, device=lens.device) < lens[:, None])[:, None, :]


def _plain(st):
    case, op = st["case"], st["op"]
    if op in ("decode", "acc"):
        if case.get("bits", 4) == 4:
            k, v = (_unpack(st[x + "_codes"], st[x + "_scales"]) for x in "kv")
        else:
            k, v = st["k"].float(), st["v"].float()
        o, lse, p = _attend(st["q"], k, v, st["lens"])
        if op == "decode":
            return o, lse
        acc = torch.where(_written(st["lens"], case["cap"]), st["acc"] + p.sum(2), st["acc_out"])
        return o, lse, acc
    if op == "append":
        b, t, at = st["at"]
        for x in "kv":
            c, scales = _quantise(st[x][b, :, t])
            codes = _pack(c)
            st[x + "_codes"][b, :, at] = codes
            st[x + "_scales"][b, :, at] = scales
            st[x + "_read"][b, :, t] = _unpack(codes, scales).to(BF16)
        return tuple(st[x + y] for x in "kv" for y in ("_read", "_scales"))
    if op == "load":
        n = case["hi"]
        keep = _written(st["lens"], n)[..., None]
        return tuple(torch.where(keep, _unpack(st[x + "_codes"][:, :, :n], st[x + "_scales"][:, :, :n]).to(BF16), st[x + "_out"]) for x in "kv")
    if op == "prompt":
        B, H, n_q, d = st["q"].shape
        Hkv, n = st["k"].shape[1:3]
        s = st["q"].float().view(B, Hkv, -1, d) @ st["k"].float().transpose(-1, -2)
        s = s.mul_(1 / math.sqrt(d)).sub_(st["lse"].view(B, Hkv, -1, 1))
        if case["causal"]:
            at = torch.arange(n_q, device=s.device)[:, None] + (n - n_q)
            s.view(B, H, n_q, n).masked_fill_(torch.arange(n, device=s.device) > at, -math.inf)
        return st["acc"] + s.exp_().sum(2)
    # evict: the last `recent` rows, then the largest weights, the lower row where two are equal
    lens, n = st["lens"][:, None, None], case["budget"]
    at = torch.arange(case["cap"], device=lens.device)
    rank = torch.where(at >= lens - case["recent"], math.inf, st["acc"])
    rank = torch.where(at < lens, rank, -math.inf)
    first = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :n]
    left = torch.arange(n, device=lens.device) < lens
    kept = torch.where(left, first, case["cap"]).sort(-1)[0]
    src = kept.clamp_max(case["cap"] - 1)
    keep, new = torch.where(left, kept, -1).to(torch.int32), st["lens"].clamp_max(n)
    acc = torch.where(left, st["acc"].gather(-1, src), 0.0)
    rows = lambda t: t.gather(2, src.view(*src.shape, *[1] * (t.dim() - 3)).expand(*src.shape, *t.shape[3:]))  # noqa: E731
    if case["bits"] == 16:
        out = [torch.where(left[..., None], rows(st[x]), st[x + "_out"]) for x in "kv"]
    else:
        for x in "kv":
            c, s = rows(st[x + "_codes"]), rows(st[x + "_scales"])
            st[x + "_codes_out"].copy_(torch.where(left[..., None], c, st[x + "_codes_out"]))
            st[x + "_scales_out"].copy_(torch.where(left[..., None, None], s, st[x + "_scales_out"]))
        out = [torch.where(left[..., None], _unpack(st[x + "_codes_out"], st[x + "_scales_out"]).to(BF16), st[x + "_out"]) for x in "kv"]
    return (keep, new, acc, *out)


# ------------------------------------------------------------------------------------------ the framework's calls
def _cache(sdpa, st, end=""):
    return sdpa.Kv4Cache(*(st[x + y + end] for x in "kv" for y in ("_codes", "_scales")))


def _own(st):
    import memory_optimal_sdpa_b200 as sdpa
    case, op = st["case"], st["op"]
    if op == "decode":
        return sdpa.decode_kv4(st["q"], _cache(sdpa, st), st["lens"])
    if op == "acc":
        if case["bits"] == 4:
            o, lse = sdpa.decode_kv4(st["q"], _cache(sdpa, st), st["lens"], acc=st["acc"], acc_out=st["acc_out"])
        else:
            o, lse = sdpa.decode_acc(st["q"], st["k"], st["v"], st["lens"], st["acc"], acc_out=st["acc_out"])
        return o, lse, st["acc_out"]
    if op == "append":
        sdpa.kv4_append(_cache(sdpa, st), st["k"], st["v"], st["lens"], n_new=st["n_new"], k_read=st["k_read"], v_read=st["v_read"])
        return tuple(st[x + y] for x in "kv" for y in ("_read", "_scales"))
    if op == "load":
        return sdpa.kv4_load(_cache(sdpa, st), st["lens"], k=st["k_out"], v=st["v_out"])
    if op == "prompt":
        return sdpa.fwd_acc(st["q"], st["k"], st["lse"], st["acc"], causal=case["causal"], acc_out=st["acc_out"])
    if case["bits"] == 16:
        keep, new = sdpa.evict(st["k"], st["v"], st["acc"], st["lens"], case["budget"], recent=case["recent"], k_out=st["k_out"], v_out=st["v_out"], acc_out=st["acc_out"])
    else:
        out = _cache(sdpa, st, "_out")
        keep, new = sdpa.kv4_evict(_cache(sdpa, st), st["acc"], st["lens"], case["budget"], recent=case["recent"], out=out, acc_out=st["acc_out"])
        sdpa.kv4_load(out, new, k=st["k_out"], v=st["v_out"])
    return keep, new, st["acc_out"], st["k_out"], st["v_out"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    B, H, d = _dims(case)
    row4 = d // 2 + d // 8  # a row's codes, and four bytes a group
    row16 = 2 * d
    if op == "prompt":
        Hkv, n_q, n = case["heads_kv"], case["n_q"], case["n_kv"]
        pairs = n_q * (n - n_q) + n_q * (n_q + 1) // 2 if case["causal"] else n_q * n
        return {"bytes": B * (H * n_q * (row16 + 4) + Hkv * n * (row16 + 8)), "flops": 2.0 * d * B * H * pairs}
    lens = _spread(case["lo"], case["hi"], B)
    if op in ("decode", "acc"):
        Hkv = case["heads_kv"]
        row = 2 * (row4 if case.get("bits", 4) == 4 else row16) + (8 if op == "acc" else 0)
        return {"bytes": sum(lens) * Hkv * row + B * H * (2 * row16 + 4), "flops": 4.0 * d * H * sum(lens)}
    if op == "append":
        rows = sum(_spread(case["rows_lo"], case["rows"], B)) * H
        return {"bytes": max(1, rows * 2 * (2 * row16 + row4)), "flops": 6.0 * d * rows}
    if op == "load":
        rows = sum(lens) * H
        return {"bytes": max(1, rows * 2 * (row16 + row4)), "flops": 4.0 * d * rows}
    kept = sum(min(n, case["budget"]) for n in lens) * H
    move = 2 * 2 * row16 if case["bits"] == 16 else 2 * (2 * row4 + row16)
    return {"bytes": sum(lens) * H * 4 + kept * (move + 8), "flops": 0.0}


# ------------------------------------------------------------------------------------------ the definitions, in 64 bits
def _value64(codes, scales, b, h):
    """Rows of one sequence and head of a 4-bit cache, channel by channel."""
    d = codes.shape[-1] * 2
    ng = d // 32
    ch = torch.arange(d, device=codes.device)
    g, r, e, high = ch // 32, ch % 32 // 4, ch % 4 // 2, ch % 2
    byte = codes[b, h][:, 2 * (r * ng + g) + e].int()
    code = torch.where(high > 0, byte.bitwise_right_shift(4), byte.bitwise_and(15))
    s = scales[b, h].double()
    return s[:, g, 0] * code + s[:, g, 1]


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    B, H, d = _dims(case)
    if op == "prompt":
        if work(case)["flops"] > 4e12:
            return None
        Hkv, n_q, n = case["heads_kv"], case["n_q"], case["n_kv"]
        out = st["acc"].double()
        key = torch.arange(n, device=out.device)
        for b in range(B):
            for h in range(H):
                for i in range(0, n_q, 1024):
                    x = torch.einsum("id,jd->ij", st["q"][b, h, i:i + 1024].double(), st["k"][b, h // (H // Hkv)].double()) / d ** 0.5
                    w = torch.exp(x - st["lse"][b, h, i:i + 1024, None].double())
                    if case["causal"]:
                        w *= key[None] - (n - n_q) <= torch.arange(i, i + len(w), device=w.device)[:, None]
                    out[b, h // (H // Hkv)] += w.sum(0)
        return out
    lens = st["lens"].tolist()
    bits4 = case.get("bits", 4) == 4
    if op in ("decode", "acc"):
        Hkv, G = case["heads_kv"], H // case["heads_kv"]
        o, lse = (torch.zeros(s, dtype=F64, device=st["q"].device) for s in ((B, H, d), (B, H)))
        acc = st["acc_out"].double() if op == "acc" else None
        for b, n in enumerate(lens):
            if n == 0:
                lse[b] = -math.inf
                continue
            for h in range(Hkv):
                k, v = ((_value64(st[x + "_codes"][:, :, :n], st[x + "_scales"][:, :, :n], b, h) if bits4 else st[x][b, h, :n].double()) for x in "kv")
                x = torch.einsum("gd,jd->gj", st["q"][b, h * G:h * G + G].double(), k) / d ** 0.5
                lse[b, h * G:h * G + G] = torch.logsumexp(x, 1)
                w = torch.softmax(x, 1)
                o[b, h * G:h * G + G] = torch.einsum("gj,jd->gd", w, v)
                if acc is not None:
                    acc[b, h, :n] = st["acc"][b, h, :n].double() + w.sum(0)
        return (o, lse) if acc is None else (o, lse, acc)
    if op == "append":
        res = []
        for x in "kv":
            read, scales = st[x + "_read"].double(), st[x + "_scales"].double()
            for b, n in enumerate(st["n_new"].tolist()):
                g = st[x][b, :, :n].double().reshape(H, n, d // 32, 32)
                if n == 0:
                    continue
                lo, step = g.min(-1).values, (g.max(-1).values - g.min(-1).values) / 15
                # bf16 values have eight significant bits: the scale is the smallest of them that is not below
                unit = torch.exp2(torch.floor(torch.log2(step.clamp_min(2.0 ** -126))) - 7)
                s = torch.ceil(step / unit) * unit
                code = torch.round((g - lo[..., None]) / torch.where(s > 0, s, 1.0)[..., None])
                read[b, :, :n] = (s[..., None] * code + lo[..., None]).reshape(H, n, d)
                scales[b, :, lens[b]:lens[b] + n] = torch.stack((s, lo), -1)
            res += [read, scales]
        return tuple(res)
    if op == "load":
        k, v = st["k_out"].double(), st["v_out"].double()
        for b, n in enumerate(lens):
            for h in range(H):
                for x, to in (("k", k), ("v", v)):
                    to[b, h, :n] = _value64(st[x + "_codes"][:, :, :n], st[x + "_scales"][:, :, :n], b, h)
        return k, v
    n = case["budget"]
    keep = torch.full((B, H, n), -1, dtype=torch.int32)
    acc = torch.zeros((B, H, n), dtype=F64, device=st["acc"].device)
    k, v = st["k_out"].double(), st["v_out"].double()
    for b, m in enumerate(lens):
        for h in range(H):
            old = max(0, m - case["recent"])
            w = st["acc"][b, h, :old].tolist()
            best = sorted(range(old), key=lambda j: (-w[j], j))[:max(0, min(m, n) - (m - old))]
            rows = sorted(best + list(range(old, m)))
            keep[b, h, :len(rows)] = torch.tensor(rows, dtype=torch.int32)
            at = torch.tensor(rows, dtype=torch.long, device=acc.device)
            acc[b, h, :len(rows)] = st["acc"][b, h, at].double()
            for x, to in (("k", k), ("v", v)):
                to[b, h, :len(rows)] = _value64(st[x + "_codes"], st[x + "_scales"], b, h)[at] if bits4 else st[x][b, h, at].double()
    return keep.to(acc.device), torch.tensor([min(m, n) for m in lens], dtype=torch.int32, device=acc.device), acc, k, v
