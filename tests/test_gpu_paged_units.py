"""The paged attention's ways of dividing its work: kv heads that share a unit
or not, units that one or many CTAs hold, layouts of the scales, scales far
apart, many sequences, calls that overlap, captured calls, and its bounded waits."""
import math

import pytest
import torch

import exact_io_aware_online_b200 as fa

from paged_ref import Cache, attend, check, quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_online_b200 import _build
    _build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def randn(shape, seed, spread=1.0):
    return (torch.randn(shape, generator=torch.Generator("cpu").manual_seed(seed)) * spread).to(torch.bfloat16)


def run(c, q, causal=True, window=-1, **kw):
    args, scales = c.cuda()
    o, lse = fa.fwd_paged(q.cuda(), *args, c.seqlens.cuda(), causal=causal, window=window, **scales, **kw)
    torch.cuda.synchronize()
    return o, lse


def compare(c, q, causal=True, window=-1, **kw):
    o, lse = run(c, q, causal, window, **kw)
    want_o, want_l, tol_o, tol_l = attend(c, q, causal, window, kw.get("scale"))
    check("O", o, want_o, tol_o)
    check("LSE", lse, want_l, tol_l)


# lengths that leave every kind of unit: none, one key, part of a tile, several tiles, many CTAs
LENS = [0, 1, 31, 33, 700, 64, 1500, 129]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("Hkv,g,Nq,d", [(4, 2, 1, 128), (8, 1, 1, 64), (8, 8, 1, 128), (12, 3, 2, 64), (2, 8, 2, 128), (6, 4, 3, 64),
                                        (4, 16, 1, 128), (8, 4, 4, 128), (3, 8, 1, 128), (1, 16, 4, 64), (1, 1, 1, 128)])
def test_heads_of_a_unit(kind, layout, Hkv, g, Nq, d):
    """Enough sequences for units of several kv heads, and kv heads that do not divide."""
    lens = LENS * (-(-64 // (Hkv * len(LENS)))) if Hkv > 1 else LENS
    c = Cache(lens, Hkv, d, 16, kind, layout, seed=201).fill_random(202)
    compare(c, randn((len(lens), Hkv * g, Nq, d), 203, 2.0))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [1, 3, 8, 12, 24, 40])
def test_pages_that_are_no_multiple_of_anything(kind, page):
    c = Cache([1, 50, 300], 4, 64, page, kind, "nhd", seed=211).fill_random(212)
    compare(c, randn((3, 8, 2, 64), 213, 2.0))
    compare(c, randn((3, 8, 2, 64), 214, 2.0), window=37)
    compare(c, randn((3, 8, 2, 64), 215, 2.0), causal=False, window=5)


def test_many_new_tokens():
    """More rows than a unit holds: blocks of 64, the last one ragged, some rows before the first token."""
    for kind in ("bf16", "e4m3"):
        c = Cache([150, 40, 0], 2, 64, 16, kind, "hnd", seed=221).fill_random(222)
        compare(c, randn((3, 6, 45, 64), 223, 2.0))
        compare(c, randn((3, 6, 45, 64), 224, 2.0), causal=False, window=9)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_thousands_of_sequences(kind):
    g = torch.Generator().manual_seed(231)
    lens = torch.randint(0, 9, (5000,), generator=g).tolist()
    c = Cache(lens, 1, 64, 4, kind, "nhd", seed=232).fill_random(233)
    compare(c, randn((5000, 1, 1, 64), 234))


def test_scales_far_apart():
    """Value rows whose sizes differ by up to 2^40, rows of zeros, and a key of the
    largest weight whose value is tiny: each output within the bound its own values give."""
    c = Cache([300, 140, 90], 4, 128, 16, "e4m3", "nhd", seed=241).fill_random(242)
    for b, n in enumerate(c.lens):
        for at in range(0, n, 7):
            c.put("v", b, torch.tensor([at]), randn((1, 4, 128), 243 + at, 2.0 ** (-(at % 41))))
        c.put("v", b, torch.tensor([n // 2]), torch.zeros((1, 4, 128), dtype=torch.bfloat16))
    c.put("k", 1, torch.tensor([11]), randn((1, 4, 128), 244, 6.0))
    c.put("v", 1, torch.tensor([11]), randn((1, 4, 128), 245, 2.0 ** -30))
    c.put("v", 2, torch.tensor([89]), randn((1, 4, 128), 246, 2.0 ** 60))
    compare(c, randn((3, 8, 2, 128), 247, 3.0))
    zero = Cache([200], 4, 128, 16, "e4m3", "nhd", seed=248)
    for at in range(200):
        zero.put("k", 0, torch.tensor([at]), randn((1, 4, 128), 249 + at))
    o, lse = run(zero, randn((1, 4, 1, 128), 250))
    assert (o == 0).all() and torch.isfinite(lse).all()


def test_queries_of_any_size():
    """The quantised path scales queries to f16's range: rows from 2^-120 to 2^100."""
    c = Cache([70, 20], 2, 64, 16, "e4m3", "nhd", seed=251).fill_random(252)
    q = randn((2, 4, 1, 64), 253)
    q[0, 0] *= 2.0 ** -120
    q[0, 1] = 0
    q[0, 2, 0, 5] = 2.0 ** 10
    compare(c, q)
    big = Cache([70, 20], 2, 64, 16, "e4m3", "nhd", seed=254)
    for b, n in enumerate(big.lens):
        for name, spread in (("k", 2.0 ** -100), ("v", 1.0)):
            big.put(name, b, torch.arange(n), randn((n, 2, 64), 255 + b, spread))
    compare(big, (randn((2, 4, 1, 64), 257).float() * 2.0 ** 100).to(torch.bfloat16))


@pytest.mark.parametrize("Hkv", [4, 8])
def test_layouts_of_the_scales(Hkv):
    """Tokens or heads in line, padded rows, and a base that is aligned to four bytes only."""
    B, P, page, d = 16, 60, 16, 64
    c = Cache([100, 3] * 8, Hkv, d, page, "e4m3", "nhd", seed=261).fill_random(262)
    q = randn((B, Hkv, 1, d), 263)
    want_o, want_l, tol_o, tol_l = attend(c, q, True, -1)
    (k, v, table), scales = c.cuda()
    P = k.shape[0]

    def padded(x, shape, order, skip):
        flat = torch.full((math.prod(shape) + skip,), math.nan, device="cuda")[skip:].view(shape).permute(order)
        flat = flat[:P, :Hkv, :page]
        flat.copy_(x)
        return flat
    for shape, order, skip in (((P, Hkv, page), (0, 1, 2), 0), ((P, Hkv, page + 3), (0, 1, 2), 1), ((P, page, Hkv), (0, 2, 1), 0),
                               ((P, page, Hkv), (0, 2, 1), 1), ((P, page + 1, Hkv + 1), (0, 2, 1), 0), ((P, page, Hkv + 4), (0, 2, 1), 4),
                               ((page, Hkv, P), (2, 1, 0), 0)):
        ks, vs = (padded(scales[n], shape, order, skip) for n in ("k_scale", "v_scale"))
        o, lse = fa.fwd_paged(q.cuda(), k, v, table, c.seqlens.cuda(), ks, vs, causal=True)
        check("O", o, want_o, tol_o)
        check("LSE", lse, want_l, tol_l)


def test_kv_in_one_buffer_and_other_page_orders():
    B, Hkv, page, d = 3, 4, 16, 128
    c = Cache([90, 300, 17], Hkv, d, page, "bf16", "nhd", seed=271).fill_random(272)
    q = randn((B, 8, 1, d), 273)
    want_o, want_l, tol_o, tol_l = attend(c, q, True, -1)
    (k, v, table), _ = c.cuda()
    P = k.shape[0]
    for shape, order in (((2, P, page, Hkv, d), (1, 3, 2, 4)), ((2, P, Hkv, page, d), (1, 2, 3, 4)), ((2, Hkv, P, page, d), (2, 1, 3, 4)),
                         ((2, page, Hkv, P, d), (3, 2, 1, 4)), ((2, P, page, Hkv + 1, d + 8), (1, 3, 2, 4))):
        both = torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda")
        kk, vv = (both[i].permute([o - 1 for o in order])[:, :Hkv, :, :d] for i in range(2))
        kk.copy_(k), vv.copy_(v)
        o, lse = fa.fwd_paged(q.cuda(), kk, vv, table, c.seqlens.cuda(), causal=True)
        check("O", o, want_o, tol_o)
        check("LSE", lse, want_l, tol_l)


def test_calls_that_overlap():
    """Two streams, a workspace each; both equal the same calls one after the other."""
    cs = [Cache([4000, 700, 5], 4, 128, 16, kind, "nhd", seed=281 + i).fill_random(283 + i) for i, kind in enumerate(("bf16", "e4m3"))]
    qs = [randn((3, 8, 1, 128), 285 + i).cuda() for i in range(2)]
    on = [c.cuda() for c in cs]
    lens = [c.seqlens.cuda() for c in cs]

    def go(i):
        (k, v, table), scales = on[i]
        return fa.fwd_paged(qs[i], k, v, table, lens[i], causal=True, **scales)
    want = [go(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(go(i))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_captured_behind_copies_and_other_streams():
    """In a graph the calls follow a copy, a memset and a kernel of another stream, and see what those left."""
    c = Cache([200, 90], 2, 128, 16, "e4m3", "nhd", seed=291).fill_random(292)
    (k, v, table), scales = c.cuda()
    new = randn((2, 2, 128), 293).cuda()
    q0 = randn((2, 4, 1, 128), 294).cuda()
    kn, q, L = torch.zeros_like(new), torch.zeros_like(q0), torch.zeros(2, dtype=torch.int32, device="cuda")
    lens, one = c.seqlens.cuda(), torch.arange(3, dtype=torch.int32, device="cuda")
    back = torch.full((2, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((2, 4, 1), device="cuda")
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            q.copy_(q0)
        L.zero_()
        L.copy_(lens)
        kn.copy_(new)
        fa.cache_write(kn, kn, k, v, table, one, L, **scales)
        main.wait_stream(side)
        fa.fwd_paged(q, k, v, table, L, causal=True, out=out, lse=lse, **scales)
        back.zero_()
        fa.cache_read(k, v, table, one, L, 2, out=(back, torch.empty_like(back)), **scales)
        kn.zero_()                                             # the write has read it
        q.zero_()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for b, n in enumerate(c.lens):
        for name in ("k", "v"):
            c.put(name, b, torch.tensor([n - 1]), new[b:b + 1].cpu())
    want_o, want_l, tol_o, tol_l = attend(c, q0.cpu(), True, -1)
    for _ in range(3):
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        check("O", out, want_o, tol_o)
        check("LSE", lse, want_l, tol_l)
        code, scale = quantise(new.cpu())
        assert torch.equal(back.cpu(), (code.float() * scale[..., None]).to(torch.bfloat16))


def test_a_step_with_nothing_to_write():
    """Sequences without new tokens (a padded batch) keep theirs."""
    c = Cache([20, 0, 33], 2, 64, 16, "bf16", "nhd", seed=301).fill_random(302)
    (k, v, table), _ = c.cuda()
    before = k.clone()
    x = randn((4, 2, 64), 303).cuda()
    cu = torch.tensor([1, 1, 1, 1], dtype=torch.int32, device="cuda")
    fa.cache_write(x, x, k, v, table, cu, c.seqlens.cuda())
    assert torch.equal(k, before)
    compare(c, randn((3, 2, 1, 64), 304))


@pytest.mark.parametrize("Hkv,lens", [(4, [3000] * 20), (1, [3000, 40])])
def test_a_stalled_load_is_reported(Hkv, lens):
    """Loads that never begin: the waits run out, the call comes back, the status
    says so, and the next call is right."""
    c = Cache(lens, Hkv, 64, 16, "e4m3", "nhd", seed=311).fill_random(312)
    q = randn((len(lens), Hkv, 1, 64), 313)
    assert fa.device_status() == 0
    fa.debug_set_wait_limit(20_000_000)
    fa.debug_set_stall(True)
    try:
        run(c, q)
        assert fa.device_status() == 6
    finally:
        fa.debug_set_stall(False)
        fa.debug_set_wait_limit(0)
    assert fa.device_status() == 0
    compare(c, q)


@pytest.mark.parametrize("kind,d,Hkv,B,longest", [("bf16", 128, 8, 20, 512), ("e4m3", 64, 4, 112, 256), ("bf16", 64, 1, 130, 700)])
def test_units_of_several_tiles_that_are_not_shared(kind, d, Hkv, B, longest):
    """Tables of at most eight tiles, and about as many sequences as groups of CTAs:
    every unit stays with one group, some groups have none, empty sequences between."""
    g = torch.Generator().manual_seed(321)
    lens = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    lens[0], lens[1], lens[-1] = 0, longest, 0
    c = Cache(lens, Hkv, d, 16, kind, "nhd", seed=322).fill_random(323)
    compare(c, randn((B, Hkv, 1, d), 324))
    empty = Cache([0] * B, Hkv, d, 16, kind, "nhd", seed=325, width=longest // 16)
    o, lse = run(empty, randn((B, Hkv, 1, d), 326))
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_sequences_that_share_pages(kind):
    """A common beginning kept once: several sequences name its pages, and the same page twice."""
    c = Cache([96, 16, 130, 0], 2, 64, 16, kind, "nhd", seed=331).fill_random(332)
    table = torch.full((4, 9), -1, dtype=torch.int32)
    table[0, :6], table[2, :9] = c.table[0, :6], c.table[2, :9]
    table[1, :4] = torch.tensor([table[0, 0], table[0, 1], table[0, 1], table[2, 0]])
    table[3, :7] = torch.cat([table[0, :6], c.table[1, :1]])
    c.table, c.lens = table, [96, 60, 130, 100]
    c.seqlens = torch.tensor(c.lens, dtype=torch.int32)
    compare(c, randn((4, 4, 2, 64), 333, 2.0))
    (k, v, tab), scales = c.cuda()
    cu = torch.tensor([0, 96, 156, 286, 386], dtype=torch.int32, device="cuda")
    rk, _ = fa.cache_read(k, v, tab, cu, c.seqlens.cuda(), 386, **scales)
    assert torch.equal(rk[286:382], rk[:96]) and torch.equal(rk[96:112], rk[:16]) and torch.equal(rk[112:128], rk[128:144])
