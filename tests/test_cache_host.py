"""The bounded decode cache on the host: exported symbols, refused arguments of the C ABI and of the binding (CPU)."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")
sdpa = pytest.importorskip("memory_optimal_sdpa_b200")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sdpa_cache.h")
P = 0x10000  # an aligned, never-dereferenced stand-in address
FAR = 1 << 40
bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
NAN, INF = float("nan"), float("inf")


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(sdpa_\w+)\s*\(", text)))


def test_header_and_library_agree():
    names = declared_functions()
    assert names == sorted(["sdpa_kv4_append", "sdpa_kv4_load", "sdpa_decode_kv4", "sdpa_decode_kv4_workspace_size",
                            "sdpa_decode_acc", "sdpa_decode_acc_workspace_size", "sdpa_fwd_acc", "sdpa_evict",
                            "sdpa_kv4_evict"])
    lib = ctypes.CDLL(sdpa.LIB_PATH)
    for name in names:
        assert hasattr(lib, name), name


def test_header_compiles_as_c(tmp_path):
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "sdpa_cache.h"\nint main(void) { return SDPA_OK; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                   check=True)


# ------------------------------------------------------------------------------------------ C ABI
def append(K=P, V=P, lens=P, n_new=None, kc=P, ks=P, vc=P, vs=P, kr=None, vr=None, b=1, h=1, n=1, cap=8, d=64):
    return sdpa.lib.sdpa_kv4_append(K, V, lens, n_new, kc, ks, vc, vs, kr, vr, b, h, n, cap, d, None)


def load(kc=P, ks=P, vc=P, vs=P, lens=P, K=P, V=P, b=1, h=1, n=1, cap=8, d=64):
    return sdpa.lib.sdpa_kv4_load(kc, ks, vc, vs, lens, K, V, b, h, n, cap, d, None)


def decode4(Q=P, kc=P, ks=P, vc=P, vs=P, lens=P, O=P, LSE=None, acc=None, out=None, b=1, hq=2, hkv=1, cap=8, d=64,
            scale=0.1, ws=P, nbytes=1 << 30):
    return sdpa.lib.sdpa_decode_kv4(Q, kc, ks, vc, vs, lens, O, LSE, acc, out, b, hq, hkv, cap, d, scale, ws, nbytes, None)


def decode16(Q=P, K=P, V=P, lens=P, O=P, LSE=None, acc=None, out=P, b=1, hq=2, hkv=1, cap=8, d=64, scale=0.1, ws=P,
             nbytes=1 << 30):
    return sdpa.lib.sdpa_decode_acc(Q, K, V, lens, O, LSE, acc, out, b, hq, hkv, cap, d, scale, ws, nbytes, None)


def fwd_acc(Q=P, K=P, LSE=P, acc=None, out=P, b=1, hq=2, hkv=1, nq=4, nkv=8, nacc=8, d=64, scale=0.1, causal=0):
    return sdpa.lib.sdpa_fwd_acc(Q, K, LSE, acc, out, b, hq, hkv, nq, nkv, nacc, d, scale, causal, None)


def evict(K=P, V=FAR, acc=2 * FAR, lens=3 * FAR, ko=4 * FAR, vo=5 * FAR, ao=6 * FAR, keep=7 * FAR, new=8 * FAR, b=1, h=1,
          cap=8, out=8, d=64, budget=4, recent=1):
    return sdpa.lib.sdpa_evict(K, V, acc, lens, ko, vo, ao, keep, new, b, h, cap, out, d, budget, recent, None)


def evict4(kc=P, ks=FAR, vc=2 * FAR, vs=3 * FAR, acc=4 * FAR, lens=5 * FAR, kco=6 * FAR, kso=7 * FAR, vco=8 * FAR,
           vso=9 * FAR, ao=10 * FAR, keep=11 * FAR, new=12 * FAR, b=1, h=1, cap=8, out=8, d=64, budget=4, recent=1):
    return sdpa.lib.sdpa_kv4_evict(kc, ks, vc, vs, acc, lens, kco, kso, vco, vso, ao, keep, new, b, h, cap, out, d, budget,
                                   recent, None)


CALLS = [append, load, decode4, decode16, fwd_acc, evict, evict4]
NULLS = {append: "K V lens kc ks vc vs", load: "K V lens kc ks vc vs", decode4: "Q kc ks vc vs lens O",
         decode16: "Q K V lens O out", fwd_acc: "Q K LSE out", evict: "K V acc lens ko vo ao keep new",
         evict4: "kc ks vc vs acc lens kco kso vco vso ao keep new"}
ALIGNED16 = {append: "K V kc ks vc vs", load: "K V kc ks vc vs", decode4: "Q kc ks vc vs O ws", decode16: "Q K V O ws",
             fwd_acc: "Q K", evict: "K V ko vo", evict4: "kc ks vc vs kco kso vco vso"}
ALIGNED4 = {append: "lens n_new", load: "lens", decode4: "lens LSE out", decode16: "lens LSE acc out",
            fwd_acc: "LSE acc out", evict: "acc lens ao keep new", evict4: "acc lens ao keep new"}


@pytest.mark.parametrize("call", CALLS)
def test_null_and_misaligned_pointers(call):
    for name in NULLS[call].split():
        assert call(**{name: None}) == sdpa.SDPA_ERR_INVALID_ARG, name
    for name in ALIGNED16[call].split():
        assert call(**{name: 20 * FAR + 8}) == sdpa.SDPA_ERR_MISALIGNED, name
    for name in ALIGNED4[call].split():
        assert call(**{name: 20 * FAR + 2}) == sdpa.SDPA_ERR_MISALIGNED, name


@pytest.mark.parametrize("call", CALLS)
def test_sizes(call):
    heads = "hq" if call in (decode4, decode16, fwd_acc) else "h"
    cap = "nkv" if call is fwd_acc else "cap"
    for bad in ({"b": -1}, {heads: -1}, {cap: 0}, {cap: -3}):
        assert call(**bad) == sdpa.SDPA_ERR_INVALID_ARG, bad
    for d in (0, 32, 96, 256, -64):
        assert call(d=d) == sdpa.SDPA_ERR_UNSUPPORTED, d
    assert call(b=0) == sdpa.SDPA_OK and call(**{heads: 0}) == sdpa.SDPA_OK
    if call is not fwd_acc:
        big = {"b": 65535, heads: 64, "cap": 1 << 20}
        if heads == "hq":
            big.update(hkv=64, nbytes=1 << 62)
        assert call(**big) == sdpa.SDPA_ERR_UNSUPPORTED
    else:
        assert call(b=65535, hq=64, hkv=64, nkv=1 << 20, nacc=1 << 20) == sdpa.SDPA_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", CALLS)
def test_rows_that_would_pass_32_bits_when_rounded_up(call):
    """2^31 - 8192 rows are the most: row numbers are rounded up to blocks in 32 bits."""
    most = (1 << 31) - 8192
    sizes = {"hq": 1, "nkv": most + 1, "nacc": most + 1} if call is fwd_acc else {"cap": most + 1}
    if call in (decode4, decode16):
        sizes.update(hq=1, nbytes=1 << 62)
    assert call(**sizes) == sdpa.SDPA_ERR_UNSUPPORTED


def test_other_arguments():
    inv = sdpa.SDPA_ERR_INVALID_ARG
    assert append(kr=P) == inv and append(vr=P) == inv and append(n=-1) == inv and append(n=0) == sdpa.SDPA_OK
    assert append(kr=P, vr=FAR) == inv and append(K=FAR, kr=2 * FAR, vr=FAR + 64) == inv  # over the rows being read
    assert load(n=-1) == inv and load(n=0) == sdpa.SDPA_OK
    for call in (decode4, decode16, fwd_acc):
        for s in (NAN, INF, -INF):
            assert call(scale=s) == inv
        assert call(hq=3, hkv=2) == inv and call(hkv=0) == inv
    assert decode4(acc=P) == inv  # weights in, nowhere to put them
    for call in (decode4, decode16):
        assert call(ws=None) == sdpa.SDPA_ERR_WORKSPACE and call(nbytes=16) == sdpa.SDPA_ERR_WORKSPACE
    assert fwd_acc(nacc=7) == inv and fwd_acc(causal=2) == inv and fwd_acc(nq=-1) == inv
    for call in (evict, evict4):
        assert call(budget=0) == inv and call(budget=9) == inv and call(recent=-1) == inv and call(recent=5) == inv
        assert call(out=0) == inv


def test_evict_refuses_overlapping_arrays():
    inv = sdpa.SDPA_ERR_INVALID_ARG
    assert evict(ko=P + 128) == inv           # into the middle of its own input
    assert evict(ko=P, out=9) == inv          # in place with another capacity
    assert evict(ko=FAR) == inv               # into the other array
    assert evict(ko=4 * FAR, vo=4 * FAR) == inv
    assert evict(ao=2 * FAR + 4) == inv
    assert evict(new=3 * FAR) == inv          # the lengths are still read while the new ones are written
    assert evict4(kso=2 * FAR) == inv and evict4(vco=P) == inv


def test_workspace_sizes():
    size4, size16 = sdpa.decode_kv4_workspace_size, sdpa.decode_acc_workspace_size
    for bad in ((0, 8, 8, 16, 64), (1, 0, 8, 16, 64), (1, 8, 0, 16, 64), (1, 9, 2, 16, 64), (1, 8, 8, 0, 64), (1, 8, 8, 16, 96)):
        assert size4(*bad) == 0 and size16(*bad) == 0
    for shape in ((1, 8, 8, 1, 64), (3, 20, 4, 1001, 128), (64, 64, 8, 16384, 128)):
        plain, kept = size4(*shape), size4(*shape, with_acc=True)
        assert 0 < plain and plain + shape[0] * shape[1] * 4 <= kept + 64 and kept % 16 == 0
        assert size16(*shape) > 0


# ------------------------------------------------------------------------------------------ binding
def t(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


def cache(B=2, H=2, n=8, d=64):
    return sdpa.Kv4Cache(t(B, H, n, d // 2, dtype=u8), t(B, H, n, d // 32, 2), t(B, H, n, d // 2, dtype=u8), t(B, H, n, d // 32, 2))


LENS = t(2, dtype=i32)


def test_binding_refuses_wrong_types_and_shapes():
    c, acc = cache(), t(2, 2, 8, dtype=f32)
    rows, q = t(2, 2, 3, 64), t(2, 4, 64)
    with pytest.raises(TypeError, match="cache must be a Kv4Cache"):
        sdpa.kv4_append(c[0], rows, rows, LENS)
    with pytest.raises(TypeError, match="cache.k_codes must be"):
        sdpa.kv4_load(c._replace(k_codes=c.k_scales), LENS)
    with pytest.raises(ValueError, match="cache.v_scales has shape"):
        sdpa.decode_kv4(q, c._replace(v_scales=t(2, 2, 8, 4, 2)), LENS)
    with pytest.raises(ValueError, match="cache.v_codes must be contiguous"):
        sdpa.decode_kv4(q, c._replace(v_codes=t(2, 8, 2, 32, dtype=u8).transpose(1, 2)), LENS)
    with pytest.raises(ValueError, match="v has shape"):
        sdpa.kv4_append(c, rows, t(2, 2, 4, 64), LENS)
    with pytest.raises(TypeError, match="n_new must be"):
        sdpa.kv4_append(c, rows, rows, LENS, n_new=t(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="both of k_read"):
        sdpa.kv4_append(c, rows, rows, LENS, k_read=rows)
    with pytest.raises(ValueError, match="both of k and v"):
        sdpa.kv4_load(c, LENS, k=rows)
    with pytest.raises(ValueError, match="k has shape"):
        sdpa.kv4_load(c, LENS, n_rows=4, k=rows, v=rows)
    with pytest.raises(TypeError, match="kv_lens must be"):
        sdpa.decode_kv4(q, c, LENS.long())
    with pytest.raises(ValueError, match="acc has shape"):
        sdpa.decode_kv4(q, c, LENS, acc=t(2, 2, 9, dtype=f32))
    with pytest.raises(TypeError, match="acc_out must be"):
        sdpa.decode_acc(q, t(2, 2, 8, 64), t(2, 2, 8, 64), LENS, acc, acc_out=acc.to(bf))
    with pytest.raises(ValueError, match="give acc"):
        sdpa.decode_acc(q, t(2, 2, 8, 64), t(2, 2, 8, 64), LENS)
    with pytest.raises(ValueError, match="lse has shape"):
        sdpa.fwd_acc(t(2, 4, 3, 64), rows, t(2, 4, 4, dtype=f32))
    with pytest.raises(ValueError, match="k_out has shape"):
        sdpa.evict(t(2, 2, 8, 64), t(2, 2, 8, 64), acc, LENS, 4, k_out=t(2, 2, 8, 128), v_out=t(2, 2, 8, 128), acc_out=acc)
    with pytest.raises(ValueError, match="acc_out together"):
        sdpa.evict(t(2, 2, 8, 64), t(2, 2, 8, 64), acc, LENS, 4, acc_out=acc)
    with pytest.raises(ValueError, match="acc_out together"):
        sdpa.kv4_evict(c, acc, LENS, 4, out=cache())
    with pytest.raises(ValueError, match="d must be 64 or 128"):
        sdpa.kv4_cache(1, 1, 8, 96, device="cpu")


def test_binding_refuses_host_tensors():
    c, acc = cache(), t(2, 2, 8, dtype=f32)
    rows, q, kv = t(2, 2, 3, 64), t(2, 4, 64), t(2, 2, 8, 64)
    for call in (lambda: sdpa.kv4_append(c, rows, rows, LENS), lambda: sdpa.kv4_load(c, LENS),
                 lambda: sdpa.decode_kv4(q, c, LENS), lambda: sdpa.decode_acc(q, kv, kv, LENS, acc),
                 lambda: sdpa.fwd_acc(t(2, 4, 3, 64), rows, t(2, 4, 3, dtype=f32)),
                 lambda: sdpa.evict(kv, kv, acc, LENS, 4), lambda: sdpa.kv4_evict(c, acc, LENS, 4)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
