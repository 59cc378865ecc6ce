"""CPU checks of the serving entry points: refusals before any CUDA call, workspace sizes, the rotation's
frequencies, and the binding's own checks."""
import ctypes
import math

import pytest

import exact_attention_140_b200 as ea

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
P = 1 << 20  # aligned address, never followed


def cache(**kw):
    a = dict(k_pages=P, v_pages=P, k_exp=None, v_exp=None, n_pages=8, page_size=16, Hkv=2, d=128, dtype=0)
    a.update(kw)
    return ea._CacheStruct(*a.values())


def rope(**kw):
    a = dict(q_weight=P, k_weight=P, freqs=P, eps=1e-6, amplitude=1.0, rot_dim=64, interleaved=0)
    a.update(kw)
    return ea._RopeStruct(*a.values())


def test_status_name():
    assert ea.attn_status_string(6) != "unknown status" and ea.STATUS[6] == "ATTN_ERR_DEVICE_INDEX"


CACHES = [(dict(n_pages=-1), INVALID), (dict(Hkv=0), INVALID), (dict(dtype=5), INVALID), (dict(page_size=8), INVALID),
          (dict(page_size=48), INVALID), (dict(page_size=8192), INVALID), (dict(d=96), UNSUPPORTED),
          (dict(Hkv=70000), UNSUPPORTED), (dict(k_pages=None), INVALID), (dict(v_pages=P + 8), MISALIGNED),
          (dict(dtype=1), INVALID), (dict(k_exp=P, v_exp=P), INVALID), (dict(dtype=1, k_exp=P), INVALID)]


def qk(**kw):
    a = dict(q=P, k=P, qo=P, ko=P, T=4, Hq=4, Hkv=2, d=128, qs=512, ks=256, qos=512, kos=256, pos=P, r=rope())
    a.update(kw)
    return ea.attn_qk_norm_rope(a["q"], a["k"], a["qo"], a["ko"], a["T"], a["Hq"], a["Hkv"], a["d"], a["qs"], a["ks"],
                                a["qos"], a["kos"], a["pos"], a["r"], stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(d=96), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(ko=None), INVALID), (dict(qs=504), INVALID), (dict(qs=516), MISALIGNED),
    (dict(k=P + 2), MISALIGNED), (dict(pos=None), INVALID), (dict(pos=P + 4), MISALIGNED), (dict(r=None), INVALID),
    (dict(r=rope(rot_dim=24)), INVALID), (dict(r=rope(rot_dim=144)), INVALID), (dict(r=rope(rot_dim=-16)), INVALID),
    (dict(r=rope(freqs=None)), INVALID), (dict(r=rope(eps=-1.0)), INVALID), (dict(r=rope(eps=math.nan)), INVALID),
    (dict(r=rope(amplitude=math.inf)), INVALID), (dict(r=rope(interleaved=2)), INVALID),
    (dict(r=rope(q_weight=P + 8)), MISALIGNED), (dict(T=0), OK), (dict(Hq=0, Hkv=0), OK)])
def test_qk_norm_rope_refusals(kw, status):
    assert qk(**kw) == status


def write(c=None, **kw):
    a = dict(k=P, v=P, T=4, ks=256, vs=256, slots=P, r=rope(), pos=P, q=P, qo=P, Hq=4, qs=512, qos=512)
    a.update(kw)
    return ea.attn_kv_write(cache() if c is None else c, a["k"], a["v"], a["T"], a["ks"], a["vs"], a["slots"], a["r"],
                            a["pos"], a["q"], a["qo"], a["Hq"], a["qs"], a["qos"], stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(r=None), INVALID), (dict(k=None), INVALID),
    (dict(slots=None), INVALID), (dict(slots=P + 4), MISALIGNED), (dict(vs=128), INVALID), (dict(ks=260), MISALIGNED),
    (dict(q=None), INVALID), (dict(qo=P + 8), MISALIGNED), (dict(pos=None), INVALID), (dict(T=0), OK)])
def test_kv_write_refusals(kw, status):
    assert write(**kw) == status


@pytest.mark.parametrize("kw,status", CACHES)
def test_cache_refusals(kw, status):
    c = cache(**kw)
    assert write(c) == status
    assert ea.attn_kv_read(c, P, 4, P, 1, P, P, 8, stream=0, raise_on_error=False) == status
    assert paged(c) == status
    assert ea.attn_fwd_paged_workspace_bytes(c, 2, 1, 2, 4, 64) == -1


def test_kv_read_refusals():
    f = lambda **kw: ea.attn_kv_read(cache(), kw.get("table", P), kw.get("width", 4), kw.get("cu", P), kw.get("n", 1),
                                     kw.get("k", P), P, kw.get("T", 8), stream=0, raise_on_error=False)
    assert f(T=-1) == INVALID and f(n=-1) == INVALID and f(width=-1) == INVALID
    assert f(cu=None) == INVALID and f(k=None) == INVALID and f(table=None) == INVALID
    assert f(k=P + 8) == MISALIGNED and f(cu=P + 2) == MISALIGNED
    assert f(T=0) == OK and f(n=0) == OK


def varlen(**kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, Tq=10, Tk=10, n=2, cq=P, ck=P, Hq=4, Hkv=2, d=128, qs=512, ks=256, vs=256,
             causal=1, scale=0.1, ws=P, wsb=1 << 20)
    a.update(kw)
    return ea.attn_fwd_varlen(a["q"], a["k"], a["v"], a["o"], a["lse"], a["Tq"], a["Tk"], a["n"], a["cq"], a["ck"],
                              a["Hq"], a["Hkv"], a["d"], a["qs"], a["ks"], a["vs"], a["causal"], a["scale"], a["ws"],
                              a["wsb"], stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(Tq=-1), INVALID), (dict(Tk=-1), INVALID), (dict(n=-1), INVALID), (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID),
    (dict(causal=2), INVALID), (dict(scale=math.nan), INVALID), (dict(d=80), UNSUPPORTED), (dict(Hq=65536 * 2), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(o=None), INVALID), (dict(cq=None), INVALID),
    (dict(n=200, Tq=300, ws=None), INVALID), (dict(n=200, Tq=300, wsb=16), INVALID),
    (dict(n=200, Tq=300, ws=P + 8), MISALIGNED), (dict(o=P + 8), MISALIGNED),
    (dict(lse=P + 2), MISALIGNED), (dict(cq=P + 1), MISALIGNED), (dict(qs=100), INVALID), (dict(ks=260), MISALIGNED),
    (dict(Tq=(1 << 31) - 1, n=(1 << 31) - 1), UNSUPPORTED),
    (dict(Tq=0), OK), (dict(n=0), OK), (dict(Hq=0), OK)])
def test_varlen_refusals(kw, status):
    assert varlen(**kw) == status


def test_varlen_workspace():
    f = ea.attn_fwd_varlen_workspace_bytes
    assert f(-1, 1, 4, 2, 128) == f(8, 1, 3, 2, 128) == f(8, 1, 4, 0, 128) == f(8, 1, 4, 2, 96) == -1
    assert f(0, 1, 4, 2, 128) == f(8, 0, 4, 2, 128) == 0
    assert f((1 << 31) - 1, (1 << 31) - 1, 4, 2, 128) == -1  # more blocks than one call takes
    assert f(1000, 128, 32, 8, 128) == (32 * ((4000 + 128 * 255) // 256) + 255) // 256 * 256
    assert f(1000, 2, 32, 8, 128) == 0  # at most a block per SM: each finds its own item
    # otherwise a list of 32-byte items: blocks of 256 rows (128 at other head sizes), groups of 4 stacked
    assert f(1000, 150, 32, 8, 128) == (32 * ((4000 + 150 * 255) // 256) + 255) // 256 * 256
    assert f(1000, 150, 8, 8, 256) == (32 * ((1000 + 150 * 127) // 128) + 255) // 256 * 256
    assert f(100000, 2, 8, 8, 128) == (32 * ((100000 + 2 * 255) // 256) + 255) // 256 * 256
    assert f(200, 500, 8, 8, 128) == (32 * ((200 + 200 * 255) // 256) + 255) // 256 * 256  # a sequence per token


def paged(c=None, **kw):
    a = dict(q=P, o=P, lse=P, Tq=4, n=2, max_q=2, cq=P, table=P, width=4, lens=P, max_kv=64, Hq=4, qs=512, causal=1,
             scale=0.1, ws=P, wsb=1 << 30)
    a.update(kw)
    return ea.attn_fwd_paged(a["q"], cache() if c is None else c, a["o"], a["lse"], a["Tq"], a["n"], a["max_q"], a["cq"],
                             a["table"], a["width"], a["lens"], a["max_kv"], a["Hq"], a["qs"], a["causal"], a["scale"],
                             a["ws"], a["wsb"], stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(Tq=-1), INVALID), (dict(n=-1), INVALID), (dict(Hq=3), INVALID), (dict(max_q=0), INVALID),
    (dict(max_q=5), INVALID), (dict(max_kv=-1), INVALID), (dict(max_kv=65), INVALID), (dict(width=-1), INVALID),
    (dict(causal=3), INVALID), (dict(scale=math.inf), INVALID), (dict(cq=None, Tq=3), INVALID),
    (dict(lens=None), INVALID), (dict(o=None), INVALID), (dict(table=None), INVALID), (dict(q=None), INVALID),
    (dict(q=P + 8), MISALIGNED), (dict(qs=516), MISALIGNED), (dict(o=P + 8), MISALIGNED), (dict(table=P + 2), MISALIGNED),
    (dict(ws=None, width=400, max_kv=6400), INVALID), (dict(wsb=100, width=400, max_kv=6400), INVALID),
    (dict(ws=P + 4, width=400, max_kv=6400), MISALIGNED),
    (dict(Tq=0), OK), (dict(n=0), OK), (dict(Hq=0), OK)])
def test_paged_refusals(kw, status):
    assert paged(**kw) == status


def test_paged_workspace():
    f = ea.attn_fwd_paged_workspace_bytes
    c = cache(Hkv=8)
    assert f(c, 0, 1, 1, 32, 64) == 0 and f(c, 4, 4, 1, 33, 64) == -1 and f(c, 4, 4, 5, 32, 64) == -1
    assert f(c, (1 << 31) - 1, (1 << 31) - 1, 32, 32, 64) == -1  # more blocks than one call takes
    assert f(c, 4, 4, 1, 32, 192) == 0  # a cluster of blocks per sequence and head
    # a count per sequence, and two partial blocks of 8 rows for each of the 50 * 8 * 3 units, or
    # of the 2 blocks that an SM holds where those are fewer
    assert f(c, 50, 50, 1, 32, 192) == 512 + 2 * 296 * 8 * 128 * 4 + 2 * 296 * 8 * 4
    assert f(c, 64, 64, 1, 32, 1 << 17) == f(c, 64, 64, 1, 32, 1 << 20)  # the grid is bounded by the GPU
    # 300 tokens of 4 stacked heads: with long contexts partial rows of several key windows
    assert f(c, 300, 1, 300, 32, 500) == 0
    assert f(c, 300, 1, 300, 32, 1 << 16) > 300 * 32 * 128 * 4 * 2


def freqs(*a, **kw):
    return ea.attn_rope_freqs(*a, **kw)


def test_rope_freqs():
    n, base = 128, 10000.0
    plain, amp = freqs(n, base)
    assert amp == 1.0 and len(plain) == 64
    for i, f in enumerate(plain):
        assert abs(f - base ** (-2 * i / n)) <= 1e-14 * f
    lin, amp = freqs(n, base, 1, 4.0)
    assert amp == 1.0 and all(abs(a * 4 - b) <= 1e-15 * b for a, b in zip(lin, plain))
    ntk, _ = freqs(n, base, 2, 8.0)
    assert ntk[0] == 1.0 and abs(ntk[-1] * 8 / plain[-1] - 1) < 1e-12  # the slowest stretched by the factor
    bands, amp = freqs(n, base, 3, 16.0, 4096.0)
    assert abs(amp - (1 + 0.1 * math.log(16))) < 1e-6
    for f, b in zip(plain, bands):
        turns = 4096 * f / (2 * math.pi)
        assert f / 16 * (1 - 1e-12) <= b <= f * (1 + 1e-12)
        if turns > 33.0 * 1.2:
            assert b == f
        if turns < 1 / 1.2:
            assert abs(b * 16 / f - 1) < 1e-12
    assert all(a > b for a, b in zip(bands, bands[1:]))
    assert freqs(n, base, 3, 1.0, 4096.0) == (plain, 1.0)


@pytest.mark.parametrize("a", [(0, 1e4), (7, 1e4), (64, 1.0), (64, math.nan), (64, 1e4, 4), (64, 1e4, 1, 0.5),
                               (64, 1e4, 3, 2.0, 0.0), (64, 1e4, 3, 2.0, 4096.0, 1.0, 1.0), (2, 1e4, 2, 2.0)])
def test_rope_freqs_refusals(a):
    with pytest.raises(ea.AttnError):
        ea.attn_rope_freqs(*a)


def test_rope_freqs_null():
    assert ea._lib.attn_rope_freqs(None, 64, 1e4, 0, 1.0, 0.0, 32.0, 1.0, None) == INVALID
    buf = (ctypes.c_double * 32)()
    assert ea._lib.attn_rope_freqs(buf, 64, 1e4, 0, 1.0, 0.0, 32.0, 1.0, None) == OK


def test_binding_checks():
    import torch
    bf = dict(dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ea.KVCache(torch.zeros(2, 16, 1, 64), torch.zeros(2, 16, 1, 64))
    with pytest.raises(ValueError):
        ea.KVCache(torch.zeros(2, 16, 1, 64, **bf), torch.zeros(2, 16, 2, 64, **bf))
    with pytest.raises(ValueError):
        ea.KVCache(torch.zeros(2, 16, 1, 64, dtype=torch.uint8), torch.zeros(2, 16, 1, 64, dtype=torch.uint8))
    with pytest.raises(TypeError):
        u = torch.zeros(2, 16, 1, 64, dtype=torch.uint8)
        ea.KVCache(u, u, u, u)
    with pytest.raises(ValueError):
        ea.KVCache(torch.zeros(2, 2, 16, 64, **bf).transpose(1, 2), torch.zeros(2, 2, 16, 64, **bf).transpose(1, 2))
    with pytest.raises(ValueError):
        ea.Rope(rot_dim=64)
    with pytest.raises(TypeError):
        ea.Rope(freqs=torch.zeros(32), rot_dim=64)
    with pytest.raises(TypeError):
        ea.Rope(q_weight=torch.zeros(64))
    with pytest.raises(ValueError):
        ea.Rope(q_weight=torch.zeros(64, **bf), k_weight=torch.zeros(128, **bf))
    with pytest.raises(TypeError):
        ea._rows(torch.zeros(3, 2, 64), "x")
    with pytest.raises(ValueError):
        ea._rows(torch.zeros(3, 64, 2, **bf).transpose(1, 2), "x")
    x = torch.zeros(5, 6, 64, **bf)
    assert ea._rows(x[:, 1:3], "x") == (5, 2, 64, 384) and ea._rows(x[:1, 1:3], "x") == (1, 2, 64, 128)
    with pytest.raises(TypeError):
        ea._index(torch.zeros(3), "x", torch.int32)
    with pytest.raises(ValueError):
        ea._index(torch.zeros(3, dtype=torch.int32), "x", torch.int32, 4)
