"""Attention over packed sequences and over the paged cache on the GPU, against the 64-bit form."""
import math

import pytest

pytestmark = pytest.mark.gpu


def setup():
    import torch

    import exact_attention_140_b200 as ea
    import serving_util as su
    return torch, ea, su


def rand(torch, *shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)


VARLEN = [  # Hq, Hkv, d, query lengths, key lengths (None: the same)
    (1, 1, 64, [1], None),
    (4, 2, 128, [1, 2, 127, 128, 129], None),
    (12, 12, 64, [0, 300, 0, 5, 257, 0], None),
    (8, 1, 128, [511, 33, 1], None),
    (6, 2, 128, [130, 260, 17], None),          # a group of 3: heads not stacked
    (4, 4, 256, [65, 1, 200], None),
    (32, 8, 128, [700, 64, 1300], None),
    (2, 1, 64, [40, 1, 300, 9], [700, 129, 1, 0]),   # longer, shorter and no keys: rows that see none
    (8, 2, 256, [3, 150], [400, 100]),
    (4, 1, 128, [256, 512], [1024, 512]),
    (16, 16, 128, [1] * 40, None),
    (4, 2, 64, [37, 0, 5, 130] * 10, None),
    (2, 2, 128, [3] * 128, [9] * 128),
    (4, 4, 64, [2, 70, 0, 300, 1] * 60, None),
    (8, 2, 128, [1, 33] * 70, [200, 33] * 70),
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", range(len(VARLEN)))
def test_varlen(case, causal):
    torch, ea, su = setup()
    Hq, Hkv, d, lq, lk = VARLEN[case]
    lk = lq if lk is None else lk
    Tq, Tk = sum(lq), sum(lk)
    q = rand(torch, Tq, Hq, d, seed=case)
    kv = rand(torch, Tk, 2 * Hkv, d, seed=case + 100)
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    scale = 1 / math.sqrt(d)
    o, lse = ea.attention_varlen(q, k, v, su.starts(lq), su.starts(lk), causal=causal)
    su.no_device_error(ea)
    a = b = 0
    for n, m in zip(lq, lk):
        ref = su.attention(q[a:a + n], k[b:b + m], v[b:b + m], causal, scale)
        if n:
            su.check_attention(o[a:a + n], lse[:, a:a + n], ref, d)
        a, b = a + n, b + m


def test_varlen_matches_each_sequence_alone():
    """A sequence's rows do not depend on its neighbours: the same bits packed and by itself."""
    torch, ea, su = setup()
    lens = [333, 1, 640, 128]
    x = rand(torch, sum(lens), 12, 128, seed=4)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    o, lse = ea.attention_varlen(q, k, v, su.starts(lens), su.starts(lens), causal=True)
    a = 0
    for n in lens:
        s = slice(a, a + n)
        o1, l1 = ea.attention_varlen(q[s], k[s], v[s], su.i32(0, n), su.i32(0, n), causal=True)
        assert torch.equal(o1, o[s]) and torch.equal(l1, lse[:, s])
        a += n


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 2, 2), (128, 4, 1), (256, 2, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_varlen_neighbours_hold_nan(d, Hq, Hkv, causal):
    """NaN and infinities in other sequences, and in the rows of a padded batch, reach no other row; rows outside
    every sequence stay as they were."""
    torch, ea, su = setup()
    lens = [70, 33, 140, 50]
    front, back = 3, 21
    T = front + sum(lens) + back
    q, kv = rand(torch, T, Hq, d, seed=1), rand(torch, T, 2 * Hkv, d, seed=2)
    cu = su.starts(lens) + front
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[:front] = bad[front + sum(lens):] = True
    bad[front + 70:front + 103] = True  # the whole second sequence
    q[bad], kv[bad] = math.nan, math.nan
    kv[front + 80] = math.inf
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    o = torch.full((T, Hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, T), 5.0, device="cuda")
    ea.attention_varlen(q, k, v, cu, cu, causal=causal, o=o, lse=lse)
    su.no_device_error(ea)
    a = front
    for i, n in enumerate(lens):
        s = slice(a, a + n)
        if i == 1:
            assert bool(torch.isnan(o[s]).all()) and bool(torch.isnan(lse[:, s]).all())
        else:
            su.check_attention(o[s], lse[:, s], su.attention(q[s], k[s], v[s], causal, 1 / math.sqrt(d)), d)
        a += n
    assert bool((o[:front] == 5).all()) and bool((o[-back:] == 5).all())
    assert bool((lse[:, :front] == 5).all()) and bool((lse[:, -back:] == 5).all())


@pytest.mark.parametrize("scale", [0.0, -0.09, 0.7])
def test_varlen_scales_without_lse(scale):
    torch, ea, su = setup()
    q, k, v = (rand(torch, 200, 2, 128, seed=i) for i in range(3))
    cu = su.i32(0, 90, 200)
    o = ea.attention_varlen(q, k, v, cu, cu, causal=True, scale=scale, return_lse=False)
    for s in (slice(0, 90), slice(90, 200)):
        su.check_attention(o[s], None, su.attention(q[s], k[s], v[s], True, scale), 128)


def test_varlen_bad_boundaries_stay_inside():
    """Boundaries outside the tensor or out of order are clamped and reported."""
    torch, ea, su = setup()
    q, k, v = (rand(torch, 100, 2, 64, seed=i) for i in range(3))
    for cu in (su.i32(0, 50, 400), su.i32(-9, 50, 100), su.i32(0, 60, 40)):
        ea.attention_varlen(q, k, v, cu, cu, causal=True)
        assert ea.attn_get_last_device_error()[0] == 6
    good = su.i32(0, 50, 100)
    o, lse = ea.attention_varlen(q, k, v, good, good, causal=True)
    su.no_device_error(ea)
    su.check_attention(o[:50], lse[:, :50], su.attention(q[:50], k[:50], v[:50], True, 0.125), 64)


PAGED = [  # Hq, Hkv, d, new tokens, cached tokens, page size
    (1, 1, 64, [1], [1], 16),
    (32, 8, 128, [1, 1, 1], [1000, 16, 17], 16),
    (32, 8, 128, [1] * 5, [64, 63, 65, 4000, 1], 64),
    (12, 12, 64, [1, 1], [333, 129], 32),
    (8, 1, 256, [1, 1], [700, 50], 16),
    (6, 2, 128, [1, 1], [257, 90], 16),            # a group of 3
    (32, 1, 128, [1, 2], [900, 300], 128),         # 64 rows of one group
    (4, 2, 128, [5, 1, 0, 3], [40, 1, 77, 3], 16),  # several new tokens, one sequence without
    (8, 8, 64, [17, 40], [800, 40], 256),
    (8, 2, 128, [300, 129, 1], [900, 129, 2000], 16),   # chunks
    (8, 2, 128, [300, 129, 1], [900, 129, 2000], 256),
    (16, 16, 64, [100, 260], [1500, 260], 64),
    (4, 1, 256, [90, 33], [500, 600], 32),
    (6, 2, 128, [200, 70], [650, 1100], 128),
    (4, 2, 64, [60, 50], [20, 0], 16),             # rows that see no key
    (2, 1, 128, [70], [4100], 4096),
]


@pytest.mark.parametrize("wide", [0, 1])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", range(len(PAGED)))
def test_paged(case, e4m3, causal, wide):
    """Every unwritten slot of the cache holds NaN, and unused table entries hold no page.  wide: a table with
    room for far longer sequences, which the sizes that steer the split are taken from."""
    torch, ea, su = setup()
    Hq, Hkv, d, new, lens, page = PAGED[case]
    cache, table, ks, vs = su.make_cache(ea, lens, page, Hkv, d, e4m3, seed=case, width=20000 // page if wide else None)
    q = rand(torch, sum(new), Hq, d, seed=case + 50)
    o = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, sum(new)), 9.0, device="cuda")
    ea.attention_paged(q, cache, table, su.i32(*lens), cu_q=su.starts(new), max_q=max(new), causal=causal,
                       o=o, lse=lse)
    su.no_device_error(ea)
    a = 0
    for n, k, v in zip(new, ks, vs):
        s = slice(a, a + n)
        if n:
            su.check_attention(o[s], lse[:, s], su.attention(q[s], k, v, causal, 1 / math.sqrt(d)), d)
        a += n


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [1, 7, 130])
def test_paged_uniform_and_bounds(n, e4m3):
    """Without boundaries every sequence has the same number of rows; a tighter max_kv changes the windows only."""
    torch, ea, su = setup()
    lens = [200, 513, 140]
    cache, table, ks, vs = su.make_cache(ea, lens, 16, 2, 128, e4m3, seed=n, width=64)
    q = rand(torch, 3 * n, 8, 128, seed=n)
    for max_kv in (None, 513):
        o, lse = ea.attention_paged(q, cache, table, su.i32(*lens), max_kv=max_kv)
        su.no_device_error(ea)
        for i in range(3):
            s = slice(i * n, i * n + n)
            su.check_attention(o[s], lse[:, s], su.attention(q[s], ks[i], vs[i], True, 1 / math.sqrt(128)), 128)


@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("e4m3", [False, True])
def test_paged_bad_indices(n, e4m3):
    """A page outside the cache reads as zeros, lengths outside their arrays are clamped; both are reported."""
    torch, ea, su = setup()
    cache, table, ks, vs = su.make_cache(ea, [256, 200], 16, 2, 64, e4m3, seed=3)
    q = rand(torch, 2 * n, 4, 64, seed=8)
    bad = table.clone()
    bad[0, 3] = 1 << 30
    o, lse = ea.attention_paged(q, cache, bad, su.i32(256, 200))
    assert ea.attn_get_last_device_error()[0] == 6
    k0, v0 = ks[0].clone(), vs[0].clone()
    k0[48:64] = v0[48:64] = 0
    su.check_attention(o[:n], lse[:, :n], su.attention(q[:n], k0, v0, True, 0.125), 64)
    su.check_attention(o[n:], lse[:, n:], su.attention(q[n:], ks[1], vs[1], True, 0.125), 64)
    o, lse = ea.attention_paged(q, cache, table, su.i32(100000, 200))  # longer than the table: its 256 keys
    assert ea.attn_get_last_device_error()[0] == 6
    su.check_attention(o[:n], lse[:, :n], su.attention(q[:n], ks[0], vs[0], True, 0.125), 64)
    o, lse = ea.attention_paged(q, cache, table, su.i32(-1, 200))
    assert ea.attn_get_last_device_error()[0] == 6
    assert bool((o[:n] == 0).all()) and bool((lse[:, :n] == -math.inf).all())


def test_paged_nan_row_is_nan():
    """A cached row that was written as NaN (exponent 255) makes the rows that see it NaN and no others."""
    torch, ea, su = setup()
    for n in (1, 70):
        cache, table, ks, vs = su.make_cache(ea, [100 + n, 150 + n], 16, 1, 128, True, seed=2)
        cache.tensors[2][table[0, 2].item(), 3, 0] = 255
        q = rand(torch, 2 * n, 2, 128, seed=1)
        o, lse = ea.attention_paged(q, cache, table, su.i32(100 + n, 150 + n))
        assert bool(torch.isnan(o[:n]).all()) and bool(torch.isnan(lse[:, :n]).all())
        su.check_attention(o[n:], lse[:, n:], su.attention(q[n:], ks[1], vs[1], True, 1 / math.sqrt(128)), 128)


def test_paged_large_scores():
    """Scores of some hundreds: the running reference moves, one key takes each row."""
    torch, ea, su = setup()
    cache, table, ks, vs = su.make_cache(ea, [600], 16, 2, 128, False, seed=9)
    for n in (1, 200):
        q = (rand(torch, n, 8, 128, seed=n).float() * 30).to(torch.bfloat16)
        o, lse = ea.attention_paged(q, cache, table, su.i32(600))
        su.check_attention(o, lse, su.attention(q, ks[0], vs[0], True, 1 / math.sqrt(128)), 128)


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt_then_steps(e4m3):
    """As a program uses them: a prompt in two chunks, then single tokens, each written and attended, against the
    attention of the whole sequence over the cached values."""
    torch, ea, su = setup()
    Hq, Hkv, d, page = 8, 2, 128, 16
    total = [150, 61]  # tokens of the two sequences in the end
    freqs, amp = ea.rope_freqs(d, 10000.0)
    w = (1 + 0.1 * torch.randn(d, device="cuda")).to(torch.bfloat16)
    rope = ea.Rope(freqs=freqs, rot_dim=d, amplitude=amp, q_weight=w, k_weight=w)
    shape = (20, page, Hkv, d)
    if e4m3:
        cache = ea.KVCache(*(torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)),
                           *(torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2)))
    else:
        cache = ea.KVCache(*(torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    table = torch.randperm(20, device="cuda").to(torch.int32)[:20].view(2, 10)
    x = [rand(torch, n, Hq + 2 * Hkv, d, seed=n) for n in total]
    have, outs, qs = [0, 0], [[], []], [[], []]
    for new in ([100, 40], [46, 17], [1, 1], [1, 1], [1, 1], [1, 1]):
        part = torch.cat([x[i][have[i]:have[i] + n] for i, n in enumerate(new)])
        pos = torch.cat([torch.arange(have[i], have[i] + n, device="cuda") for i, n in enumerate(new)])
        seq = torch.repeat_interleave(torch.arange(2, device="cuda"), torch.tensor(new, device="cuda"))
        slots = table[seq, pos // page].long() * page + pos % page
        q = ea.kv_write(cache, part[:, Hq:Hq + Hkv], part[:, Hq + Hkv:], slots, q=part[:, :Hq], positions=pos, rope=rope)
        have = [h + n for h, n in zip(have, new)]
        o, _ = ea.attention_paged(q, cache, table, su.i32(*have), cu_q=su.starts(new), max_q=max(new))
        for i, s in enumerate((slice(0, new[0]), slice(new[0], None))):
            outs[i].append(o[s])
            qs[i].append(q[s])
    su.no_device_error(ea)
    assert have == total
    k, v = ea.kv_read(cache, table, su.starts(total), sum(total))
    a = 0
    for i, n in enumerate(total):
        s = slice(a, a + n)
        q = torch.cat(qs[i])
        ref = su.attention(q, k[s], v[s], True, 1 / math.sqrt(d))
        su.check_attention(torch.cat(outs[i]), None, ref, d)
        o, _ = ea.attention_varlen(q, k[s].contiguous(), v[s].contiguous(), su.i32(0, n), su.i32(0, n), causal=True)
        su.check_attention(o, None, ref, d)
        a += n
    if not e4m3:  # what went in came back: the separate pass gives the same keys
        rk = torch.cat([ea.qk_norm_rope(x[i][:, :Hq], x[i][:, Hq:Hq + Hkv], torch.arange(n, device="cuda"), rope)[1]
                        for i, n in enumerate(total)])
        assert torch.equal(rk, k)


@pytest.mark.parametrize("many", [1, 30])
def test_graph_replayed_with_other_lengths(many):
    """Lengths, boundaries and pages are read on the device: one captured step serves later ones (small calls, and
    calls whose work is listed, shared between blocks and merged by further kernels)."""
    torch, ea, su = setup()
    Hq, Hkv, d = 8, 2, 128
    n = 5 * many
    cache, table, ks, vs = su.make_cache(ea, [300] * n, 16, Hkv, d, True, seed=1)
    lens, cu = su.i32(*[300] * n), su.starts([1] * n)
    q = rand(torch, n, Hq, d, seed=1)
    cq = su.starts([60] * n)
    T = 60 * n
    x = rand(torch, T, 4, 64, seed=2)
    chunk = rand(torch, 4 * n, 24, 128, seed=3)  # max_q 8: 96 rows of a key/value head at most, so the block kernel
    cc = su.starts([4] * n)

    def step():
        return (ea.attention_paged(q, cache, table, lens, cu_q=cu, max_q=1),
                ea.attention_varlen(x[:, :2], x[:, 2:3], x[:, 3:], cq, cq, causal=True),
                ea.attention_paged(chunk, cache, table, lens, cu_q=cc, max_q=8))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (o, lse), (o2, l2), (o3, l3) = step()
    for new, c in (([300] * 5, [0, 100, 260, 260, 280, 300]), ([7, 160, 299, 8, 50], [0, 259, 260, 261, 262, 263]),
                   ([1, 0, 64, 300, 128], [0, 30, 200, 201, 250, 251])):
        new, c = new * many, [i + 300 * m for m in range(many) for i in c[:-1]] + [300 * (many - 1) + c[-1]]
        lens.copy_(su.i32(*new))
        cq.copy_(su.i32(*c))
        graph.replay()
        su.no_device_error(ea)
        for i in range(0, n, 1 if many == 1 else 7):
            m, scale = new[i], 1 / math.sqrt(d)
            su.check_attention(o[i:i + 1], lse[:, i:i + 1], su.attention(q[i:i + 1], ks[i][:m], vs[i][:m], True, scale), d)
            s = slice(4 * i, 4 * i + 4)
            su.check_attention(o3[s], l3[:, s], su.attention(chunk[s], ks[i][:m], vs[i][:m], True, scale), d)
            s = slice(c[i], c[i + 1])
            if s.stop > s.start:
                su.check_attention(o2[s], l2[:, s], su.attention(x[s, :2], x[s, 2:3], x[s, 3:], True, 0.125), 64)


@pytest.mark.parametrize("n", [3, 60, 150])
def test_calls_on_two_streams(n):
    """Calls with workspaces of their own may overlap."""
    torch, ea, su = setup()
    lens = ([900, 1200, 40] * n)[:n]
    cache, table, ks, vs = su.make_cache(ea, lens, 16, 2, 128, n != 60, seed=4)
    q = rand(torch, n, 8, 128, seed=5)
    kv = su.i32(*lens)
    want = ea.attention_paged(q, cache, table, kv)
    x = rand(torch, 50 * n, 6, 128, seed=6)
    cu = su.starts([50] * n)
    want2 = ea.attention_varlen(x[:, :4], x[:, 4:5], x[:, 5:], cu, cu, causal=True)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(12):
        got.append(ea.attention_paged(q, cache, table, kv, stream=s[i % 2]))
        got.append(ea.attention_varlen(x[:, :4], x[:, 4:5], x[:, 5:], cu, cu, causal=True, stream=s[1 - i % 2]))
    torch.cuda.synchronize()
    su.no_device_error(ea)
    for i in range(0, 24, 2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want))
        assert all(torch.equal(a, b) for a, b in zip(got[i + 1], want2))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens", [[1] * 3, [64, 128, 129, 1], [3000] * 40 + [5] * 60, [0, 0, 7], [33000, 12], [500] * 300])
def test_decoding_lengths(lens, e4m3):
    """One token of every sequence: lengths at the borders of units, one long sequence shared by all blocks, many
    short ones in a block's run, and sequences without a key."""
    torch, ea, su = setup()
    cache, table, ks, vs = su.make_cache(ea, lens, 32, 2, 64, e4m3, seed=len(lens))
    n = len(lens)
    q = rand(torch, n, 12, 64, seed=7)
    o, lse = ea.attention_paged(q, cache, table, su.i32(*lens))
    su.no_device_error(ea)
    for i in range(0, n, 1 if n < 10 else 11):
        su.check_attention(o[i:i + 1], lse[:, i:i + 1], su.attention(q[i:i + 1], ks[i], vs[i], True, 0.125), 64)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.08, 0.6])
@pytest.mark.parametrize("n", [1, 3, 90])
def test_paged_scales(n, scale, e4m3):
    torch, ea, su = setup()
    cache, table, ks, vs = su.make_cache(ea, [400], 64, 2, 128, e4m3, seed=6)
    q = rand(torch, n, 8, 128, seed=n)
    o, lse = ea.attention_paged(q, cache, table, su.i32(400), scale=scale)
    su.check_attention(o, lse, su.attention(q, ks[0], vs[0], True, scale), 128)


def test_scales_of_far_apart_powers():
    """Value rows of an e4m3 cache whose scales differ by 2^30 to 2^90."""
    torch, ea, su = setup()
    cache, table, ks, vs = su.make_cache(ea, [500], 16, 1, 128, True, seed=6)
    k_exp, v_exp = cache.tensors[2], cache.tensors[3]
    ids = table[0].long()
    i = torch.arange(500, device="cuda")
    e = torch.where(i % 3 == 0, 60, torch.where(i % 3 == 1, 120, 150)).to(torch.uint8)  # 2^-67, 2^-7, 2^23
    v_exp[ids[i // 16], i % 16, 0] = e
    v = cache.tensors[1][ids[i // 16], i % 16].view(torch.float8_e4m3fn).double() * su.pow2(e.long() - 127)[:, None, None]
    for n in (1, 100):
        q = rand(torch, n, 4, 128, seed=n)
        o, lse = ea.attention_paged(q, cache, table, su.i32(500))
        su.check_attention(o, lse, su.attention(q, ks[0], v, True, 1 / math.sqrt(128)), 128)


def test_queries_of_far_apart_sizes():
    """f16 products over an e4m3 cache: query rows from 1e-30 to 1e30, and elements of one row that differ by 2^30."""
    torch, ea, su = setup()
    cache, table, ks, vs = su.make_cache(ea, [300] * 4, 16, 1, 128, True, seed=8)
    q = rand(torch, 4, 4, 128, seed=3).float()
    q[0] *= 1e-30
    q[1] *= 1e-3
    q[1, :, ::2] *= 2.0 ** -30
    q[2, 0] = 0
    q = q.to(torch.bfloat16)
    o, lse = ea.attention_paged(q, cache, table, su.i32(300, 300, 300, 300))
    for i in range(4):
        su.check_attention(o[i:i + 1], lse[:, i:i + 1],
                           su.attention(q[i:i + 1], ks[i], vs[i], True, 1 / math.sqrt(128)), 128)
    big = (rand(torch, 1, 4, 128, seed=3).float() * 1e30).to(torch.bfloat16)
    o, _ = ea.attention_paged(big, cache, table[:1], su.i32(300), scale=1e-31)
    su.check_attention(o, None, su.attention(big, ks[0], vs[0], True, 1e-31), 128)


@pytest.mark.parametrize("e4m3", [False, True])
def test_cache_beyond_32_bits(e4m3):
    """Pages whose elements lie past 2^31 and 2^32: write, read and both attention kernels."""
    torch, ea, su = setup()
    page, Hkv, d = 16, 8, 128
    n_pages = (1 << 32) // (page * Hkv * d) + 40
    shape = (n_pages, page, Hkv, d)
    t = [torch.empty(shape, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda") for _ in range(2)]
    e = [torch.empty(shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2)] if e4m3 else []
    cache = ea.KVCache(*t, *e)
    T = 200
    kv = rand(torch, T, 2 * Hkv, d, seed=1)
    pages = torch.tensor([n_pages - 1 - 2 * i for i in range(10)] + [n_pages // 2 + i for i in range(3)], device="cuda")
    table = pages.to(torch.int32).view(1, -1)
    i = torch.arange(T, device="cuda")
    ea.kv_write(cache, kv[:, :Hkv], kv[:, Hkv:], pages[i // page] * page + i % page)
    k, v = ea.kv_read(cache, table, su.i32(0, T), T)
    su.no_device_error(ea)
    if e4m3:
        val, ex = su.quantise(kv)
        want = val * su.pow2(ex - 127).unsqueeze(-1)
    else:
        want = kv.double()
    assert torch.equal(k.double(), want[:, :Hkv]) and torch.equal(v.double(), want[:, Hkv:])
    for n in (1, 40, 150):
        q = rand(torch, n, 16, d, seed=n)
        o, lse = ea.attention_paged(q, cache, table, su.i32(T))
        su.check_attention(o, lse, su.attention(q, k, v, True, 1 / math.sqrt(d)), d)
    del t, e, cache
    torch.cuda.empty_cache()


def test_empty_calls():
    torch, ea, su = setup()
    z = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    o, lse = ea.attention_varlen(z, z, z, su.i32(0), su.i32(0), causal=True)
    assert o.shape == (0, 4, 128) and lse.shape == (4, 0)
    q = rand(torch, 5, 4, 128, seed=1)
    o, lse = ea.attention_varlen(q, z, z, su.i32(0, 5), su.i32(0, 0), causal=False)  # queries, but no key anywhere
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    none = torch.empty(0, 16, 4, 128, dtype=torch.bfloat16, device="cuda")
    cache = ea.KVCache(none, none.clone())
    for n in (5, 1):
        o, lse = ea.attention_paged(q[:n], cache, torch.zeros(n, 3, dtype=torch.int32, device="cuda"),
                                    torch.zeros(n, dtype=torch.int32, device="cuda"))
        assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    q90 = rand(torch, 90, 4, 128, seed=1)
    o, lse = ea.attention_paged(q90, cache, torch.zeros(1, 3, dtype=torch.int32, device="cuda"), su.i32(0))
    assert bool((o == 0).all())
    ea.kv_write(cache, z, z, torch.empty(0, dtype=torch.int64, device="cuda"))
    k, _ = ea.kv_read(cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), su.i32(0, 0), 0)
    assert k.shape == (0, 4, 128)
    su.no_device_error(ea)


def test_tensors_elsewhere_are_refused():
    torch, ea, su = setup()
    q = rand(torch, 5, 4, 64, seed=1)
    with pytest.raises(ValueError):
        ea.attention_varlen(q, q.cpu(), q.cpu(), su.i32(0, 5), su.i32(0, 5))
    with pytest.raises(ValueError):
        ea.attention_varlen(q, q, q, su.i32(0, 5).cpu(), su.i32(0, 5))
    pages = torch.zeros(2, 16, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ea.attention_paged(q, ea.KVCache(pages, pages.clone()), torch.zeros(5, 1, dtype=torch.int32, device="cuda"),
                           torch.ones(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ea.qk_norm_rope(q, q, torch.arange(5, device="cuda"),
                        ea.Rope(freqs=ea.rope_freqs(64, 1e4, device="cpu")[0], rot_dim=64))
    with pytest.raises(TypeError):
        ea.attention_varlen(q.float(), q, q, su.i32(0, 5), su.i32(0, 5))
    with pytest.raises(TypeError):
        ea.attention_varlen(q, q, q, su.i32(0, 5).long(), su.i32(0, 5))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,new,cached", [(64, 1, 900), (128, 3, 700), (128, 40, 333), (128, 1024, 1500), (256, 300, 800),
                                          (256, 512, 512)])
def test_sequences_share_pages(d, new, cached, e4m3):
    """A shared prefix: sequences whose table rows name the same pages, and a page that a row names twice."""
    torch, ea, su = setup()
    page = 64
    cache, table, ks, vs = su.make_cache(ea, [cached], page, 2, d, e4m3, seed=d)
    i = torch.arange(cached, device="cuda")
    i = torch.where(i < 2 * page, i % page, i)  # the third sequence: its second page is its first again
    twice = table[:1].clone()
    twice[0, 1] = twice[0, 0]
    both = torch.cat([table[:1], table[:1], twice]).contiguous()
    q = rand(torch, 3 * new, 4, d, seed=2)
    o, lse = ea.attention_paged(q, cache, both, su.i32(cached, cached - 5, cached))
    su.no_device_error(ea)
    for s, (k, v) in enumerate([(ks[0], vs[0]), (ks[0][:-5], vs[0][:-5]), (ks[0][i], vs[0][i])]):
        r = slice(s * new, (s + 1) * new)
        su.check_attention(o[r], lse[:, r], su.attention(q[r], k, v, True, 1 / math.sqrt(d)), d)


def test_two_threads():
    """Calls from two host threads, each on a stream of its own."""
    import threading

    torch, ea, su = setup()
    cache, table, ks, vs = su.make_cache(ea, [700, 80], 32, 2, 128, True, seed=9)
    kv = su.i32(700, 80)
    x = rand(torch, 400, 8, 128, seed=1)
    cu = su.i32(0, 150, 400)

    def work():
        o, lse = ea.attention_paged(x[:2], cache, table, kv)
        c, _ = ea.attention_paged(x[:160], cache, table, kv)
        p, _ = ea.attention_varlen(x, x[:, :2], x[:, 2:4], cu, cu, causal=True)
        return o, lse, c, p

    want = work()
    torch.cuda.synchronize()
    wrong = []

    def run(stream):
        with torch.cuda.stream(stream):
            for _ in range(40):
                if not all(torch.equal(a, b) for a, b in zip(work(), want)):
                    wrong.append(stream)

    threads = [threading.Thread(target=run, args=(torch.cuda.Stream(),)) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    su.no_device_error(ea)


def test_prompt_step_captured_and_replayed():
    """Write, a long chunk over an e4m3 cache (expanded, in windows) and its single-token form in one graph; a second
    graph of the same calls replayed in turn with it."""
    torch, ea, su = setup()
    Hq, Hkv, d, page, T, cached = 8, 2, 128, 64, 300, 3000
    cache, table, ks, vs = su.make_cache(ea, [cached], page, Hkv, d, True, seed=3)
    ids = table[0].long()
    x = [rand(torch, T, Hq + 2 * Hkv, d, seed=i) for i in (1, 2)]
    pos = torch.arange(cached - T, cached, device="cuda")
    slots = ids[pos // page] * page + pos % page
    lens = su.i32(cached)

    def step(y):
        ea.kv_write(cache, y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], slots)
        return ea.attention_paged(y[:, :Hq], cache, table, lens), ea.attention_paged(y[-1:, :Hq], cache, table, lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for y in x:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(y))
        graphs.append(g)
    for which in (0, 1, 0):
        graphs[which].replay()
        su.no_device_error(ea)
        k, v = ks[0].clone(), vs[0].clone()
        for new, c in ((x[which][:, Hq:Hq + Hkv], k), (x[which][:, Hq + Hkv:], v)):
            val, ex = su.quantise(new)
            c[-T:] = val * su.pow2(ex - 127).unsqueeze(-1)
        (o, lse), (o1, l1) = outs[which]
        ref = su.attention(x[which][:, :Hq], k, v, True, 1 / math.sqrt(d))
        su.check_attention(o, lse, ref, d)
        su.check_attention(o1, l1, su.attention(x[which][-1:, :Hq], k, v, True, 1 / math.sqrt(d)), d)


PIECES = [  # Hq, Hkv, d, new tokens, cached tokens, page size
    (32, 8, 128, [256, 100, 130, 300], [6000, 2500, 4100, 300], 16),
    (24, 8, 128, [300, 70, 1], [5000, 900, 64], 64),     # a group of 3: heads not stacked
    (12, 12, 64, [700, 33, 0, 256], [4000, 50, 77, 3000], 32),
    (16, 8, 256, [200, 90], [3000, 2600], 16),
    (32, 8, 128, [513, 100, 65], [400, 20, 0], 128),     # rows that see no key, and a sequence without any
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", range(len(PIECES)))
def test_paged_pieces(case, e4m3, causal):
    """Chunks whose key tiles are cut into one equal run per SM: by a table with room for long sequences, of which
    some are short; captured, and replayed with other lengths and boundaries."""
    torch, ea, su = setup()
    Hq, Hkv, d, new, cached, page = PIECES[case]
    n, T, top = len(new), sum(new), 16384
    cache, table, ks, vs = su.make_cache(ea, cached, page, Hkv, d, e4m3, seed=case, width=top // page)
    q = rand(torch, T, Hq, d, seed=case)
    cu, lens = su.starts(new), su.i32(*cached)
    # the workspace of pieces: their list, the places of the items' tiles, two partial blocks an SM, and rows of an
    # expanded cache
    g, rows = (Hq // Hkv if Hq // Hkv != 3 else 1), 128 if d == 256 else 256
    items, nh = (T * g + n * (rows - 1)) // rows, Hkv if g > 1 else Hq
    up = lambda x, to=256: (x + to - 1) // to * to
    want = (up(up(48 * (items * nh + 148), 16) + 8 * (items + 2) + 4 * (n + 1)) + 296 * rows * d * 4 + up(296 * rows * 4))
    if e4m3 and d > 64 and max(new) * (Hq // Hkv) >= (1024 if d == 128 else 512):
        want += 2 * n * top * Hkv * d * 2
    assert ea.attn_fwd_paged_workspace_bytes(cache.struct, T, n, max(new), Hq, top) == want
    o, lse = torch.empty_like(q), torch.empty(Hq, T, device="cuda")

    def check(new, cached):
        a = 0
        for s, (i, m) in enumerate(zip(new, cached)):
            r = slice(a, a + i)
            if i:
                su.check_attention(o[r], lse[:, r], su.attention(q[r], ks[s][:m], vs[s][:m], causal, 1 / math.sqrt(d)), d)
            a += i

    def call():
        ea.attention_paged(q, cache, table, lens, cu_q=cu, max_q=max(new), causal=causal, o=o, lse=lse)

    call()
    su.no_device_error(ea)
    check(new, cached)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    other = [max(m - 37 * (s + 1), 0) for s, m in enumerate(cached)]
    moved = new[:]
    moved[0], moved[1] = new[0] - 17, new[1] + 9
    lens.copy_(su.i32(*other))
    cu.copy_(su.starts(moved))
    o.fill_(7.0)
    graph.replay()
    su.no_device_error(ea)
    check(moved, other)
    assert bool((o[sum(moved):] == 7).all())  # rows behind the last sequence


def test_pieces_of_bad_boundaries():
    """Boundaries that overlap, so that the items are more than there can be: reported, and the next call is right."""
    torch, ea, su = setup()
    new, cached = [300, 70, 200], [3000, 900, 2000]
    cache, table, ks, vs = su.make_cache(ea, cached, 32, 8, 128, False, seed=3, width=512)
    q = rand(torch, 570, 32, 128, seed=1)
    lens = su.i32(*cached)
    for cu in (su.i32(0, 570, 0, 570), su.i32(0, 700, 300, 570), su.i32(-5, 100, 570, 100)):
        ea.attention_paged(q, cache, table, lens, cu_q=cu, max_q=570)
        assert ea.attn_get_last_device_error()[0] == 6
    o, lse = ea.attention_paged(q, cache, table, lens, cu_q=su.starts(new), max_q=300)
    su.no_device_error(ea)
    su.check_attention(o[370:], lse[:, 370:], su.attention(q[370:], ks[2], vs[2], True, 1 / math.sqrt(128)), 128)
