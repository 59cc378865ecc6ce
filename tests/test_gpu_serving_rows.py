"""Norm, rotation and the paged cache's write and read on the GPU, against their 64-bit forms."""
import math

import pytest

pytestmark = pytest.mark.gpu


def setup():
    import torch

    import exact_attention_140_b200 as ea
    import serving_util as su
    return torch, ea, su


def rope_of(torch, ea, d, rot, interleaved, norm, amplitude=1.0, base=10000.0, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = [(1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(torch.bfloat16) if norm else None for _ in range(2)]
    freqs = ea.rope_freqs(rot, base)[0] if rot else None
    return ea.Rope(freqs=freqs, rot_dim=rot, interleaved=interleaved, amplitude=amplitude, q_weight=w[0], k_weight=w[1],
                   eps=1e-5), w, freqs


def rows_bound(torch, ref, x_ref, amplitude=1.0):
    """bf16's half step 2^-8 |y|, and fp32 arithmetic: a few 2^-24 of the operands of each sum (norm, cosine and
    sine from an angle reduced in fp64 to within 2^-23 turns), 2e-6 of the pair's size at most."""
    return 2.0 ** -8 * ref.abs() + 2e-6 * amplitude * x_ref.abs().amax(-1, keepdim=True) + 1e-38


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (5, 7, 3), (64, 32, 8), (700, 12, 12), (2049, 4, 1)])
@pytest.mark.parametrize("d,rot,interleaved,norm", [
    (64, 64, False, True), (64, 32, True, False), (128, 128, False, True), (128, 128, True, True),
    (128, 48, False, False), (128, 0, False, True), (256, 256, True, True), (256, 64, False, True),
    (256, 256, False, False), (128, 16, True, False)])
def test_norm_rope(T, Hq, Hkv, d, rot, interleaved, norm):
    torch, ea, su = setup()
    rope, w, freqs = rope_of(torch, ea, d, rot, interleaved, norm, amplitude=1.25)
    g = torch.Generator(device="cuda").manual_seed(T + d)
    x = torch.randn(T, Hq + 2 * Hkv, d, device="cuda", generator=g).to(torch.bfloat16)
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]  # slices of a fused projection
    pos = torch.randint(0, 1 << 20, (T,), device="cuda", generator=g)
    qo, ko = ea.qk_norm_rope(q, k, pos, rope)
    su.no_device_error(ea)
    for got, src, wt in ((qo, q, w[0]), (ko, k, w[1])):
        ref = su.norm_rope(src, wt, 1e-5, pos, freqs, rot, interleaved, 1.25)
        plain = su.norm_rope(src, wt, 1e-5, pos, freqs, 0, interleaved, 1.25)
        err = (got.double() - ref).abs()
        assert bool((err <= rows_bound(torch, ref, plain, 1.25)).all()), err.max()
    # in place on the slices: the same bits, and the values' heads untouched
    before = x[:, Hq + Hkv:].clone()
    ea.qk_norm_rope(q, k, pos, rope, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(x[:, Hq + Hkv:], before)


def test_far_and_negative_positions():
    """The angle keeps its accuracy where position * frequency passes fp32's integers."""
    torch, ea, su = setup()
    rope, _, freqs = rope_of(torch, ea, 64, 64, False, False)
    pos = torch.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 + 12345, -(2 ** 33)], device="cuda")
    q = torch.randn(6, 2, 64, device="cuda").to(torch.bfloat16)
    qo, ko = ea.qk_norm_rope(q, q[:, :1], pos, rope)
    ref = su.norm_rope(q, None, 0, pos, freqs, 64, False, 1.0)
    # (the fp64 angle itself is exact to 2^-53 of 2^33 radians: 1e-6)
    assert bool(((qo.double() - ref).abs() <= rows_bound(torch, ref, q.double()) + 2e-6 * 6).all())
    assert torch.equal(qo[:, :1], ko)


def test_norm_of_extremes():
    """Rows of zeros, and of values whose squares leave no room in bf16."""
    torch, ea, su = setup()
    rope, w, _ = rope_of(torch, ea, 128, 0, False, True)
    x = torch.zeros(3, 1, 128, device="cuda", dtype=torch.bfloat16)
    x[1] = 1e18
    x[2, 0, 5] = 1e-15
    qo, _ = ea.qk_norm_rope(x, x, None, rope)
    ref = su.norm_rope(x, w[0], 1e-5, None, None, 0, False, 1.0)
    assert bool(((qo.double() - ref).abs() <= rows_bound(torch, ref, ref)).all())
    assert bool((qo[0] == 0).all())


def test_one_side_only():
    torch, ea, su = setup()
    rope, w, freqs = rope_of(torch, ea, 128, 128, False, True)
    q = torch.randn(9, 4, 128, device="cuda").to(torch.bfloat16)
    pos = torch.arange(9, device="cuda")
    both = ea.qk_norm_rope(q, q, pos, rope)
    out = torch.empty_like(q)
    ea.attn_qk_norm_rope(q, None, out, None, 9, 4, 0, 128, 512, 0, 512, 0, pos, rope.struct)
    assert torch.equal(out, both[0])
    ea.attn_qk_norm_rope(None, q, None, out, 9, 0, 4, 128, 0, 512, 0, 512, pos, rope.struct)
    assert torch.equal(out, both[1])


def new_cache(torch, ea, n_pages, page, Hkv, d, e4m3, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if not e4m3:
        t = [torch.randn(n_pages, page, Hkv, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
        return ea.KVCache(*t)
    t = [torch.randint(0, 120, (n_pages, page, Hkv, d), device="cuda", generator=g).to(torch.uint8) for _ in range(2)]
    e = [torch.randint(100, 140, (n_pages, page, Hkv), device="cuda", generator=g).to(torch.uint8) for _ in range(2)]
    return ea.KVCache(t[0], t[1], e[0], e[1])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,Hkv,d,page,n_pages", [(1, 1, 64, 16, 2), (7, 3, 128, 16, 4), (300, 8, 128, 64, 9),
                                                 (1000, 12, 64, 32, 40), (513, 2, 256, 128, 6), (130, 1, 256, 16, 10)])
def test_write(T, Hkv, d, page, n_pages, e4m3):
    """Pure writes are exact: bf16 rows as they are, e4m3 codes and exponents as the 64-bit form rounds them;
    skipped tokens and other slots stay as they were."""
    torch, ea, su = setup()
    cache = new_cache(torch, ea, n_pages, page, Hkv, d, e4m3)
    old = [t.clone() if t is not None else None for t in cache.tensors]
    g = torch.Generator(device="cuda").manual_seed(T)
    x = (torch.randn(T, 2 * Hkv, d, device="cuda", generator=g)
         * 2.0 ** torch.randint(-30, 30, (T, 2 * Hkv, 1), device="cuda", generator=g)).to(torch.bfloat16)
    x[T // 2, 0] = 0
    slots = torch.randperm(n_pages * page, device="cuda", generator=g)[:T]
    slots[T // 3] = -5
    if T == 1:
        slots[0] = n_pages * page - 1
    ea.kv_write(cache, x[:, :Hkv], x[:, Hkv:], slots)
    su.no_device_error(ea)
    live = slots >= 0
    for i, src in ((0, x[:, :Hkv]), (1, x[:, Hkv:])):
        want = old[i].flatten(0, 1)
        if not e4m3:
            want[slots[live]] = src[live]
        else:
            val, e = su.quantise(src)
            want[slots[live]] = val[live].to(torch.float8_e4m3fn).view(torch.uint8)
            we = old[2 + i].flatten(0, 1)
            we[slots[live]] = e[live].to(torch.uint8)
            assert torch.equal(cache.tensors[2 + i].flatten(0, 1), we)
        assert torch.equal(cache.tensors[i].flatten(0, 1), want)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,interleaved", [(1, 8, 1, 128, 128, False), (64, 32, 8, 128, 128, False),
                                                       (37, 6, 3, 64, 32, True), (900, 4, 4, 256, 256, True)])
def test_write_with_rope(T, Hq, Hkv, d, rot, interleaved, e4m3):
    torch, ea, su = setup()
    rope, w, freqs = rope_of(torch, ea, d, rot, interleaved, True)
    page, n_pages = 16, T // 16 + 3
    cache = new_cache(torch, ea, n_pages, page, Hkv, d, e4m3)
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, Hq + 2 * Hkv, d, device="cuda", generator=g).to(torch.bfloat16)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    slots = torch.randperm(n_pages * page, device="cuda", generator=g)[:T]
    pos = torch.randint(0, 100000, (T,), device="cuda", generator=g)
    qo = ea.kv_write(cache, k, v, slots, q=q, positions=pos, rope=rope)
    su.no_device_error(ea)
    q_ref, k_ref = (su.norm_rope(s, wt, 1e-5, pos, freqs, rot, interleaved, 1.0) for s, wt in ((q, w[0]), (k, w[1])))
    assert bool(((qo.double() - q_ref).abs() <= rows_bound(torch, q_ref, q_ref * 2)).all())
    kp, vp = (t.flatten(0, 1)[slots] for t in cache.tensors[:2])
    if not e4m3:
        # the same arithmetic as the separate pass: the same bits
        assert torch.equal(kp, ea.qk_norm_rope(q, k, pos, rope)[1]) and torch.equal(vp, v)
        return
    ke, ve = (t.flatten(0, 1)[slots].double() for t in cache.tensors[2:])
    val, e = su.quantise(v)
    assert torch.equal(vp.view(torch.float8_e4m3fn).double(), val) and torch.equal(ve, e.double())
    scale = su.pow2(ke.long() - 127).unsqueeze(-1)
    got = kp.view(torch.float8_e4m3fn).double() * scale
    # half a step of e4m3 (2^-4 of the value; 2^-10 of the scale below its normal range) and the fp32 rows' error
    bound = 2.0 ** -4 * k_ref.abs() + 2.0 ** -10 * scale + 4e-6 * k_ref.abs().amax(-1, keepdim=True)
    assert bool(((got - k_ref).abs() <= bound).all())
    _, e_ref = su.quantise(k_ref)  # the exponent may differ only where the maximum is at a power's edge
    off = (ke - e_ref.double()).abs()
    assert off.max() <= 1 and off.mean() <= 0.01


def test_write_edges_of_the_exponent():
    torch, ea, su = setup()
    vals = [448.0, 450.0, 449.0, 224.0, 1.75, 1.7578125, 2.0 ** -126, 2.0 ** -133, 3.38953139e38, 0.0, -448.0,
            2.0 ** -109, 1.75 * 2.0 ** -109, 2.0 ** 100]
    T = len(vals)
    x = torch.zeros(T, 1, 64, device="cuda", dtype=torch.bfloat16)
    x[:, 0, 3] = torch.tensor(vals, device="cuda").to(torch.bfloat16)
    x[:, 0, 4] = x[:, 0, 3] * 0.0091
    cache = new_cache(torch, ea, 1, 16, 1, 64, True)
    slots = torch.arange(T, device="cuda")
    ea.kv_write(cache, x, x, slots)
    val, e = su.quantise(x)
    for i in range(2):
        assert torch.equal(cache.tensors[2 + i][0, :T], e.to(torch.uint8))
        assert torch.equal(cache.tensors[i][0, :T].view(torch.float8_e4m3fn).double(), val)
    k, v = ea.kv_read(cache, su.i32(0).view(1, 1), su.i32(0, T), T)
    want = val * torch.tensor([2.0 ** int(n) for n in (e - 127).flatten()], device="cuda", dtype=torch.float64).view(T, 1, 1)
    # bf16's largest value, 255/256 * 2^128, rounds to 256 * 2^120 in four bits: an infinity in bf16
    want = want.float().to(torch.bfloat16)
    assert bool(torch.isinf(want[8, 0, 3])) and int(torch.isinf(want).sum()) == 1
    assert torch.equal(k, want) and torch.equal(v, want)


def test_write_non_finite_rows_and_bad_slots():
    torch, ea, su = setup()
    cache = new_cache(torch, ea, 2, 16, 2, 128, True)
    old = [t.clone() for t in cache.tensors]
    x = torch.randn(6, 2, 128, device="cuda").to(torch.bfloat16)
    x[0, 0, 7], x[1, 1, 0], x[2, 0, 127] = math.nan, math.inf, -math.inf
    slots = torch.tensor([0, 1, 2, 32, 1 << 40, 5], device="cuda")  # two of them outside the cache
    ea.kv_write(cache, x, x, slots)
    rc, word = ea.attn_get_last_device_error()
    assert rc == 6 and word == 2
    assert ea.attn_get_last_device_error()[0] == 0
    k, _ = ea.kv_read(cache, su.i32(0).view(1, 1), su.i32(0, 6), 6)
    bad = torch.zeros(6, 2, dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[1, 1] = bad[2, 0] = True
    assert torch.equal(torch.isnan(k).all(-1), bad) and torch.equal(torch.isnan(k).any(-1), bad)
    for t, o in zip(cache.tensors, old):  # every other slot as it was
        assert torch.equal(t[0, 6:], o[0, 6:]) and torch.equal(t[1], o[1]) and torch.equal(t[0, 3:5], o[0, 3:5])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,page,Hkv,d", [([1], 16, 1, 64), ([0, 17, 16, 0, 333], 16, 3, 128), ([1000, 5], 128, 8, 128),
                                            ([70, 64, 63], 64, 2, 256), ([4097], 4096, 1, 64), ([0, 0], 16, 1, 128)])
def test_read(lens, page, Hkv, d, e4m3):
    torch, ea, su = setup()
    cache, table, ks, vs = su.make_cache(ea, lens, page, Hkv, d, e4m3, seed=sum(lens) + d)
    T = sum(lens)
    cu = su.starts(lens) + 2  # two rows in front of the first sequence, three behind the last
    k = torch.full((T + 5, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    ea.kv_read(cache, table, cu, T + 5, k_out=k, v_out=v)
    su.no_device_error(ea)
    for got, parts in ((k, ks), (v, vs)):
        assert torch.equal(got[2:2 + T].double(), torch.cat(parts))
        assert bool((got[:2] == 7).all()) and bool((got[2 + T:] == 7).all())


def test_read_every_code_and_exponent():
    torch, ea, su = setup()
    codes = torch.arange(256, device="cuda").to(torch.uint8)
    codes = torch.where((codes & 0x7F) == 0x7F, 0, codes).to(torch.uint8)
    n = 254
    pages = codes.view(4, 64).repeat(64, 1).view(16, 16, 1, 64)[:, :, :, :].contiguous()
    e = torch.arange(256, device="cuda").clamp(1, n).to(torch.uint8).view(16, 16, 1).contiguous()
    cache = ea.KVCache(pages, pages, e, e)
    table = torch.arange(16, dtype=torch.int32, device="cuda").view(1, 16)
    k, _ = ea.kv_read(cache, table, su.i32(0, 256), 256)
    val = pages.view(torch.float8_e4m3fn).double().view(256, 1, 64)
    p = torch.tensor([2.0 ** (int(x) - 127) for x in e.flatten()], dtype=torch.float64, device="cuda").view(256, 1, 1)
    # one rounding to bf16 where a subnormal or an overflow needs it
    assert torch.equal(k, (val * p).float().to(torch.bfloat16))


def test_read_bad_pages():
    torch, ea, su = setup()
    cache, table, ks, vs = su.make_cache(ea, [40], 16, 2, 64, True, seed=5)
    t = table.clone()
    t[0, 1] = cache.n_pages
    k, v = ea.kv_read(cache, t, su.i32(0, 40), 40)
    assert ea.attn_get_last_device_error()[0] == 6
    assert bool((k[16:32] == 0).all()) and torch.equal(k[:16].double(), ks[0][:16]) and torch.equal(v[32:].double(), vs[0][32:])
    ea.kv_read(cache, table, su.i32(0, 60), 60)  # more tokens than the table has pages for
    assert ea.attn_get_last_device_error()[0] == 6
