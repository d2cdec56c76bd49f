"""The 8-bit serving operators without a GPU: argument checks of the C ABI (answered before any
CUDA call) and of the Python layer, pins of the float64 oracle, and a model of how
fq_kv_append finds its work items."""

import ctypes
import math
import random

import numpy as np
import pytest
import torch

from oracle import serving as osv

_P = 0x10000  # an aligned address that no check dereferences


@pytest.fixture(scope="module")
def lib():
    from rotation_bit_quantization_token_b200 import build as b
    b.build()
    from rotation_bit_quantization_token_b200 import _lib
    return _lib.load()


def _cache(**kw):
    from rotation_bit_quantization_token_b200 import _lib
    d = dict(k=_P, v=_P, k_scale=_P, v_scale=_P, num_pages=64, kv_heads=4, page_size=32, head_dim=128)
    d.update(kw)
    return _lib.KvCacheDesc(**d)


def _batch(**kw):
    from rotation_bit_quantization_token_b200 import _lib
    d = dict(cu_new=_P, seq_lens=_P, page_table=_P, num_seqs=3, table_width=8)
    d.update(kw)
    return _lib.KvBatchDesc(**d)


BAD_CACHE = [({"k": None}, 161001), ({"v": None}, 161001), ({"k_scale": None}, 161001), ({"v_scale": None}, 161001),
             ({"k": _P + 8}, 161002), ({"num_pages": 0}, 161002), ({"num_pages": 1 << 31}, 161002),
             ({"num_pages": (1 << 31) // 128}, 161002), ({"kv_heads": 0}, 161002), ({"kv_heads": 257}, 161002),
             ({"page_size": 8}, 161002), ({"page_size": 48}, 161002), ({"page_size": 256}, 161002),
             ({"head_dim": 96}, 161002), ({"head_dim": 256}, 161002)]
BAD_BATCH = [({"cu_new": None}, 161001), ({"seq_lens": None}, 161001), ({"page_table": None}, 161001),
             ({"num_seqs": 0}, 161002), ({"num_seqs": 65537}, 161002), ({"table_width": 0}, 161002),
             ({"table_width": (1 << 24) + 1}, 161002), ({"cu_new": _P + 2}, 161002)]


def _append(lib, cache, batch, **kw):
    a = dict(T=5, dtype=0, k=_P, ks=512, v=_P, vs=512, f=_P, rot=64, il=0, q=_P, qs=1024, hq=8, qo=_P)
    a.update(kw)
    return lib.fq_kv_append(cache, batch, a["T"], a["dtype"], a["k"], a["ks"], a["v"], a["vs"], a["f"], a["rot"],
                            a["il"], a["q"], a["qs"], a["hq"], a["qo"], None, None)


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_cache_descriptor_is_checked(lib, kw, code):
    c, b = _cache(**kw), _batch()
    assert _append(lib, ctypes.byref(c), ctypes.byref(b)) == code
    n = ctypes.c_int64(7)
    assert lib.fq_kv_attention_workspace(ctypes.byref(c), ctypes.byref(b), 5, 8, 2, 100, ctypes.byref(n)) == code


@pytest.mark.parametrize("kw,code", BAD_BATCH)
def test_batch_descriptor_is_checked(lib, kw, code):
    c, b = _cache(), _batch(**kw)
    assert _append(lib, ctypes.byref(c), ctypes.byref(b)) == code
    n = ctypes.c_int64(7)
    assert lib.fq_kv_attention_workspace(ctypes.byref(c), ctypes.byref(b), 5, 8, 2, 100, ctypes.byref(n)) == code


@pytest.mark.parametrize("kw,code", [
    ({"T": 0}, 161002), ({"T": (1 << 24) + 1}, 161002), ({"dtype": 2}, 161002), ({"k": None}, 161001),
    ({"v": None}, 161001), ({"ks": 504}, 161002), ({"ks": 516}, 161002), ({"k": _P + 4}, 161002),
    ({"vs": -512}, 161002), ({"f": None}, 161001), ({"rot": 72}, 161002), ({"rot": -16}, 161002),
    ({"rot": 144}, 161002), ({"il": 2}, 161002), ({"q": None}, 161001), ({"qo": None}, 161001),
    ({"hq": 6}, 161002), ({"hq": 0}, 161002), ({"qs": 1016}, 161002), ({"qo": _P + 2}, 161002),
    ({"q": None, "qo": None}, 161001)])
def test_append_arguments_are_checked(lib, kw, code):
    c, b = _cache(), _batch()
    assert _append(lib, ctypes.byref(c), ctypes.byref(b), **kw) == code
    assert _append(lib, None, ctypes.byref(b)) == 161001
    assert _append(lib, ctypes.byref(c), None) == 161001


@pytest.mark.parametrize("kw,code", [
    ({"T": 0}, 161002), ({"dtype": 2}, 161002), ({"q": None}, 161001), ({"out": None}, 161001), ({"hq": 6}, 161002),
    ({"hq": 1028}, 161002), ({"mq": 0}, 161002), ({"mq": 6}, 161002), ({"ms": 0}, 161002), ({"ms": 257}, 161002),
    ({"scale": math.inf}, 161002), ({"scale": math.nan}, 161002), ({"causal": 2}, 161002), ({"qs": 1000}, 161002),
    ({"q": _P + 8}, 161002), ({"out": _P + 4}, 161002), ({"lse": _P + 2}, 161002), ({"ws": _P + 8}, 161002)])
def test_attention_arguments_are_checked(lib, kw, code):
    a = dict(T=5, dtype=0, q=_P, qs=1024, hq=8, mq=2, ms=256, scale=0.1, causal=1, out=_P, lse=None, ws=None, n=0)
    a.update(kw)
    c, b = _cache(), _batch()
    assert lib.fq_kv_attention(ctypes.byref(c), ctypes.byref(b), a["T"], a["dtype"], a["q"], a["qs"], a["hq"], a["mq"],
                               a["ms"], a["scale"], a["causal"], a["out"], a["lse"], a["ws"], a["n"], None, None) == code
    assert lib.fq_kv_attention_workspace(ctypes.byref(c), ctypes.byref(b), 5, 8, 2, 100, None) == 161001


@pytest.mark.parametrize("kw,code", [
    ({"a": None}, 161001), ({"sa": None}, 161001), ({"w": None}, 161001), ({"sw": None}, 161001), ({"C": None}, 161001),
    ({"T": 0}, 161002), ({"T": 262145}, 161002), ({"O": 0}, 161002), ({"O": 262145}, 161002), ({"L": 0}, 161002),
    ({"L": 24}, 161002), ({"L": 65552}, 161002), ({"t": 3}, 161002), ({"a": _P + 8}, 161002), ({"w": _P + 4}, 161002),
    ({"sa": _P + 2}, 161002), ({"C": _P + 1}, 161002), ({"st": _P + 2}, 161002)])
def test_int8_matmul_arguments_are_checked(lib, kw, code):
    a = dict(T=4, O=4, L=64, a=_P, sa=_P, w=_P, sw=_P, t=0, C=_P, st=None)
    a.update(kw)
    assert lib.fq_int8_matmul(a["T"], a["O"], a["L"], a["a"], a["sa"], a["w"], a["sw"], a["t"], a["C"], a["st"],
                              None) == code


def test_python_layer_refuses_cpu_tensors_and_wrong_shapes():
    import rotation_bit_quantization_token_b200 as fq
    a = torch.zeros(4, 64, dtype=torch.int8)
    s = torch.ones(4)
    with pytest.raises(ValueError, match="CUDA"):
        fq.int8_matmul(a, s, a, s)
    with pytest.raises(TypeError, match="Tensor"):
        fq.int8_matmul([1], s, a, s)
    k = torch.zeros(3, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.zeros(3, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        fq.KVCache.from_buffers(k, k, sc, sc)


# ---- the oracle ----

def test_oracle_e4m3_agrees_with_torch_cast():
    codes = np.arange(256, dtype=np.uint8)
    vals = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(osv.E4M3, vals, equal_nan=True)
    finite = np.abs(vals) <= 448
    assert np.array_equal(osv.e4m3_encode(vals[finite]), codes[finite])
    x = np.random.default_rng(0).standard_normal(20000) * np.exp2(np.random.default_rng(1).integers(-12, 8, 20000))
    x = np.clip(x, -448, 448).astype(np.float32)
    mids = (osv.E4M3[:126] + osv.E4M3[1:127]) / 2  # every tie
    x = np.concatenate([x, mids, -mids]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(osv.e4m3_encode(x.astype(np.float64)), want)
    assert osv.e4m3_encode(np.array([1e9, -470.0])).tolist() == [0x7E, 0xFE]


@pytest.mark.parametrize("amax,e", [(0.0, -40), (448.0, 0), (448.0001, 1), (447.9, 0), (224.0, -1), (1e-30, -40),
                                    (1e30, 40), (1.0, -8), (1.75, -8), (1.7500001, -7)])
def test_oracle_page_exponent(amax, e):
    assert osv.page_exponent(amax) == e


def test_oracle_rotary_is_a_rotation():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 2, 64))
    f = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    for il in (False, True):
        y = osv.rotary(x, np.arange(5) + 100, f, il)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 32:], x[..., 32:])
        # turning by p then by r is turning by p + r
        z = osv.rotary(y, np.full(5, 7), f, il)
        assert np.allclose(z, osv.rotary(x, np.arange(5) + 107, f, il))


def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(4)
    codes = osv.e4m3_encode(rng.standard_normal((3, 1, 16, 64)))
    sc = np.full((3, 1), 127, dtype=np.uint8)
    q = np.zeros((2, 2, 64))
    out, lse, _ = osv.kv_attention(q, codes, sc, codes, sc, [0, 2], [20], [[2, 0]], 0.125, True)
    v = osv.kv_values(codes, sc, [2, 0], 20)
    # a zero query weighs every key alike
    assert np.allclose(out[1, 0], v[:, 0].mean(0)) and np.allclose(lse[:, 0], np.log([19, 20]))
    out, lse, _ = osv.kv_attention(q, codes, sc, codes, sc, [0, 2], [1], [[2, 0]], 0.125, True)
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0])) and np.allclose(out[1, 1], v[0, 0])


def test_append_items_cover_every_touched_page_once():
    """fq_kv_append's items: start(b) = cu[b] / page + 2b, local page = item - start, for
    T / page + 2B items; every page that receives tokens is found exactly once."""
    r = random.Random(0)
    for _ in range(300):
        page = r.choice([16, 32, 64, 128])
        B = r.randint(1, 9)
        new = [r.choice([0, 1, 1, 2, r.randint(0, 400)]) for _ in range(B)]
        lens = [n + r.choice([0, r.randint(0, 300)]) for n in new]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        T = max(cu[-1], 1) + r.choice([0, 0, 3])
        start = [cu[b] // page + 2 * b for b in range(B)]
        found = []
        for item in range(T // page + 2 * B):
            b = max(x for x in range(B) if start[x] <= item)
            local = item - start[b]
            first = lens[b] - new[b]
            if new[b] > 0 and (first // page + local) * page < lens[b]:
                found.append((b, first // page + local))
        want = [(b, p) for b in range(B) if new[b] for p in range((lens[b] - new[b]) // page, (lens[b] - 1) // page + 1)]
        assert sorted(found) == want
