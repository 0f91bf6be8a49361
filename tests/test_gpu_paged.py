"""The paged key/value cache on the GPU: writing, reading back and attention,
each against the 64-bit reading in paged_ref.py, on seeded synthetic inputs."""
import math

import numpy as np
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
    return o, lse


CASES = [
    # lens, H, Hkv, Nq, d, page, kind, layout, causal, window
    ([1], 1, 1, 1, 64, 1, "bf16", "hnd", True, -1),
    ([0, 1, 2, 0], 4, 2, 1, 128, 16, "bf16", "nhd", True, -1),
    ([0, 0, 0], 4, 2, 2, 128, 16, "e4m3", "nhd", True, -1),
    ([15, 16, 17, 63, 64, 65, 127, 128, 129], 8, 2, 1, 128, 16, "bf16", "hnd", True, -1),
    ([15, 16, 17, 63, 64, 65, 127, 128, 129], 8, 2, 1, 64, 16, "e4m3", "nhd", True, -1),
    ([1000], 32, 8, 1, 128, 16, "bf16", "nhd", True, -1),
    ([3001], 4, 1, 1, 128, 128, "e4m3", "hnd", True, -1),
    ([2777, 5, 391], 16, 1, 1, 64, 48, "bf16", "hnd", True, -1),
    ([700, 33, 1], 8, 1, 1, 128, 7, "e4m3", "nhd", True, -1),             # odd pages
    ([257, 3, 900], 6, 2, 3, 128, 32, "bf16", "hnd", True, -1),           # drafts, 9 rows a kv head
    ([257, 3, 900, 2], 32, 4, 4, 64, 32, "e4m3", "nhd", True, -1),        # 32 rows
    ([190, 2, 70], 64, 1, 1, 128, 16, "e4m3", "nhd", True, -1),           # one kv head, 64 rows
    ([190, 65], 48, 1, 1, 128, 16, "bf16", "nhd", True, -1),              # 48 rows
    ([130, 4], 24, 2, 6, 64, 16, "bf16", "hnd", True, -1),                # 72 rows: more than one block
    ([130, 4], 40, 2, 5, 128, 16, "e4m3", "hnd", True, 50),               # 100 rows under a window
    ([500, 64, 10], 8, 8, 1, 64, 16, "bf16", "nhd", True, 100),           # window, one row a kv head
    ([500, 64, 10], 8, 4, 3, 128, 16, "e4m3", "nhd", True, 0),            # each row its own key
    ([500, 64, 10], 8, 4, 3, 128, 16, "bf16", "nhd", False, 7),           # band on both sides
    ([300, 1, 5], 4, 2, 4, 64, 64, "bf16", "nhd", False, -1),             # no mask; rows before the start
    ([40] * 70, 5, 5, 1, 64, 16, "bf16", "nhd", True, -1),                # many short sequences
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention_matches_the_64_bit_reading(case):
    lens, H, Hkv, Nq, d, page, kind, layout, causal, window = case
    c = Cache(lens, Hkv, d, page, kind, layout, seed=11).fill_random(12)
    compare(c, randn((len(lens), H, Nq, d), 13, 2.0), causal, window)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_large_scores_and_uneven_values(kind):
    """Scores far apart (one key takes a row) that arrive late and early, and
    value rows whose sizes differ by 2^12."""
    c = Cache([600, 90], 2, 128, 16, kind, "nhd", seed=21).fill_random(22)
    for b, pos in ((0, 3), (0, 599), (1, 40)):
        c.put("k", b, torch.tensor([pos]), randn((1, 2, 128), 23 + pos, 8.0))
        c.put("v", b, torch.tensor([pos]), randn((1, 2, 128), 24 + pos, 4096.0))
    compare(c, randn((2, 8, 2, 128), 25, 3.0))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Nq,window", [(1, -1), (3, -1), (3, 40)])
def test_nothing_masked_or_unused_is_felt(kind, Nq, window):
    """NaN in every page that no sequence uses, in the ends of pages behind the
    last token and outside the window; the newest token, which the earlier
    rows of the call may not see, is infinite and NaN."""
    lens = [130, 67, 1, 0]
    clean = Cache(lens, 2, 128, 16, kind, "nhd", seed=31).fill_random(32)
    dirty = Cache(lens, 2, 128, 16, kind, "nhd", seed=31, fill=math.nan).fill_random(32)
    for b, n in enumerate(lens):
        lo = max(0, n - Nq - window) if window >= 0 else 0
        for at in range(0, lo):
            for name in ("k", "v"):
                dirty.put(name, b, torch.tensor([at]), torch.full((1, 2, 128), math.nan, dtype=torch.bfloat16))
        if n >= Nq > 1:
            for name in ("k", "v"):
                x = randn((1, 2, 128), 33)
                x[0, 0, 5] = math.nan
                x[0, 1, 6] = math.inf
                dirty.put(name, b, torch.tensor([n - 1]), x)
    q = randn((4, 4, Nq, 128), 34)
    o, lse = run(clean, q, window=window)
    o2, lse2 = run(dirty, q, window=window)
    keep = slice(0, Nq - 1) if Nq > 1 else slice(0, 1)
    want_o, want_l, tol_o, tol_l = attend(clean, q, True, window)
    check("O", o2[:, :, keep], want_o[:, :, keep], tol_o[:, :, keep])
    check("LSE", lse2[:, :, keep], want_l[:, :, keep], tol_l[:, :, keep])
    if Nq > 1:                                             # and the row that sees it knows
        assert not torch.isfinite(o2[0, :, -1]).all()


def test_nan_values_reach_the_rows_that_see_them():
    for kind in ("bf16", "e4m3"):
        c = Cache([50, 50], 2, 64, 16, kind, "hnd", seed=35).fill_random(36)
        x = randn((1, 2, 64), 37)
        x[0, 1, 3] = math.nan
        c.put("v", 0, torch.tensor([20]), x)
        o, lse = run(c, randn((2, 4, 1, 64), 38))
        assert torch.isnan(o[0, 2:, 0, 3]).all() and torch.isfinite(o[0, :2]).all() and torch.isfinite(o[1]).all()
        assert torch.isfinite(lse).all()


def test_missing_pages_are_not_attended_to():
    c = Cache([200, 100], 2, 128, 16, "bf16", "nhd", seed=41).fill_random(42)
    c.table[0, 3], c.table[0, 12], c.table[1, 0] = -1, c.P, -(2 ** 31)
    c.table[1, 1:] = 2 ** 31 - 1                               # nothing left of sequence 1
    o, lse = compare(c, randn((2, 4, 1, 128), 43))
    assert (o[1] == 0).all() and torch.isinf(lse[1]).all()


def test_lengths_are_clamped_to_the_table():
    c = Cache([64, 64, 64], 2, 64, 16, "bf16", "nhd", seed=44).fill_random(45)
    c.seqlens = torch.tensor([2 ** 31 - 1, -5, 65], dtype=torch.int32)
    compare(c, randn((3, 4, 2, 64), 46))


def test_strided_queries_outputs_and_tables():
    c = Cache([300, 20, 77], 4, 128, 16, "e4m3", "nhd", seed=51).fill_random(52)
    qkv = randn((3, 2, 24, 128), 53).cuda()                  # [B, Nq, heads of q, k and v, d]
    q = qkv[:, :, :16].transpose(1, 2)
    out = torch.full((3, 2, 20, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    args, scales = c.cuda()
    wide = torch.full((3, args[2].shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, :args[2].shape[1]] = args[2]
    o, lse = fa.fwd_paged(q, args[0], args[1], wide[:, :args[2].shape[1]], c.seqlens.cuda(), causal=True,
                          out=out[:, :, 2:18].transpose(1, 2), **scales)
    want_o, want_l, tol_o, tol_l = attend(c, q.cpu(), True, -1)
    check("O", o, want_o, tol_o)
    check("LSE", lse, want_l, tol_l)
    assert (out[:, :, :2] == 7).all() and (out[:, :, 18:] == 7).all()
    dense, _ = fa.fwd_paged(q.contiguous(), *args, c.seqlens.cuda(), causal=True, **scales)
    assert torch.equal(dense, o)


def test_attention_is_deterministic_and_takes_a_workspace():
    c = Cache([5000, 10, 1200], 2, 128, 64, "bf16", "hnd", seed=61).fill_random(62)
    q = randn((3, 8, 1, 128), 63)
    a = run(c, q)
    size = fa.fwd_paged_workspace_size(3, 8, 2, 1, 128)
    ws = torch.full((max(size, 16) + 64,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        b = run(c, q, workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (ws[max(size, 16):] == 255).all()                                     # nothing behind its end


def test_long_ragged_batch_sampled():
    """Lengths from 1 to 20000 over many SMs, some sequences shared by dozens of
    them: sampled sequences against the 64-bit reading."""
    lens = [20000, 1, 7000, 128, 0, 13333, 64, 4097]
    c = Cache(lens, 2, 128, 64, "bf16", "nhd", seed=71).fill_random(72)
    q = randn((len(lens), 8, 1, 128), 73)
    compare(c, q)


def test_tall_caches_pass_32_bit_offsets():
    """Pages whose element offsets pass 2^32."""
    page, d, Hkv, P = 128, 128, 8, 40000                      # 5.2e9 elements
    k = torch.zeros((P, Hkv, page, d), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros((P, Hkv, page, d), dtype=torch.float8_e4m3fn, device="cuda")
    ks, vs = torch.zeros((P, Hkv, page), device="cuda"), torch.zeros((P, Hkv, page), device="cuda")
    table = torch.tensor([[P - 1, 33000, 2]], dtype=torch.int32, device="cuda")
    n = 300
    x, y = randn((n, Hkv, d), 81), randn((n, Hkv, d), 82)
    L, cu = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    fa.cache_write(x.cuda(), y.cuda(), k, v, table, cu, L, ks, vs)
    rk, rv = fa.cache_read(k, v, table, cu, L, n, ks, vs)
    for got, want in ((rk, x), (rv, y)):
        code, scale = quantise(want)
        assert torch.equal(got.cpu(), (code.float() * scale[..., None]).to(torch.bfloat16))
    c = Cache([n], Hkv, d, page, "e4m3", seed=83)
    c.put("k", 0, torch.arange(n), x)
    c.put("v", 0, torch.arange(n), y)
    q = randn((1, 16, 1, d), 84)
    o, lse = fa.fwd_paged(q.cuda(), k, v, table, L, ks, vs, causal=True)
    want_o, want_l, tol_o, tol_l = attend(c, q, True, -1)
    check("O", o, want_o, tol_o)
    check("LSE", lse, want_l, tol_l)


# ---------------------------------------------------------------- writing and reading
MOVES = [
    # new tokens a sequence, tokens before, Hkv, d, page, kind, layout
    ([1], [0], 1, 64, 1, "bf16", "hnd"),
    ([1, 1, 1, 1], [0, 15, 16, 100], 8, 128, 16, "e4m3", "nhd"),
    ([0, 3, 0, 0, 77, 1, 0], [5, 0, 0, 31, 20, 2, 9], 5, 128, 16, "bf16", "nhd"),
    ([0, 3, 0, 0, 77, 1, 0], [5, 0, 0, 31, 20, 2, 9], 5, 64, 7, "e4m3", "hnd"),
    ([200, 10], [0, 3], 2, 128, 48, "e4m3", "nhd"),
    ([9] * 80, [3] * 80, 3, 64, 8, "bf16", "nhd"),              # more than 32 sequences
    ([2] * 1100, [0] * 1100, 1, 64, 4, "e4m3", "nhd"),           # more than 1024
    ([0, 0], [4, 4], 2, 64, 4, "bf16", "hnd"),                   # no tokens at all
]


def offsets(new):
    return torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)


@pytest.mark.parametrize("case", MOVES, ids=[str(i) for i in range(len(MOVES))])
@pytest.mark.parametrize("fused", [False, True])
def test_write_and_read_back(case, fused):
    new, old, Hkv, d, page, kind, layout = case
    lens = [a + b for a, b in zip(new, old)]
    before = Cache(lens, Hkv, d, page, kind, layout, seed=91).fill_random(92)
    after = Cache(lens, Hkv, d, page, kind, layout, seed=91).fill_random(92)
    T = sum(new)
    qkv = randn((T, 3 * Hkv, d), 93, 5.0)
    k, v = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
    at = 0
    for b, n in enumerate(new):
        if n:
            for name, x in (("k", k), ("v", v)):
                after.put(name, b, torch.arange(lens[b] - n, lens[b]), x[at:at + n])
        at += n
    args, scales = before.cuda()
    dk, dv = (qkv.cuda()[:, Hkv:2 * Hkv], qkv.cuda()[:, 2 * Hkv:]) if fused else (k.contiguous().cuda(), v.contiguous().cuda())
    cu, L = offsets(new).cuda(), before.seqlens.cuda()
    fa.cache_write(dk, dv, *args, cu, L, **scales)
    torch.cuda.synchronize()
    got = {"k_pages": args[0], "v_pages": args[1]} | scales
    for name, want in after.t.items():                        # the whole pool, codes and scales bit for bit
        as_bytes = (lambda x: x.contiguous().view(torch.uint8)) if want.dtype != torch.bfloat16 else lambda x: x.contiguous().view(torch.int16)
        assert torch.equal(as_bytes(got[name].cpu()), as_bytes(want)), name

    rk, rv = fa.cache_read(*args, cu, L, T, **scales)
    full = offsets(lens).cuda()
    if fused:                                                  # heads outer in the dense buffer
        bk, bv = (torch.full((Hkv, sum(lens) + 2, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ak, av = fa.cache_read(*args, full, L, sum(lens) + 2, out=(bk.transpose(0, 1), bv.transpose(0, 1)), **scales)
    else:
        ak, av = fa.cache_read(*args, full, L, sum(lens), **scales)
    at = 0
    for name, part, whole in (("k", rk, ak), ("v", rv, av)):
        at = new_at = 0
        for b, n in enumerate(lens):
            want = torch.from_numpy(after.rows(name, b, torch.arange(n)))
            # the product code * scale is exact in 64 bits; the fp32 product's rounding can move bf16's by one
            # step only where it lands on a tie, so compare with the fp32 product
            if kind != "bf16":
                pid, slot = after.places(b, torch.arange(n))
                want = torch.stack([after.t[name + "_pages"][p, :, s].float() for p, s in zip(pid.tolist(), slot.tolist())]) \
                    * after.t[name + "_scale"][pid, :, slot][..., None] if n else want
            want = want.to(torch.bfloat16)
            assert torch.equal(whole[at:at + n].cpu(), want), (name, b)
            assert torch.equal(part[new_at:new_at + new[b]].cpu(), want[n - new[b]:]), (name, b)
            at, new_at = at + n, new_at + new[b]
        if fused:
            assert (whole[at:] == 3).all()                     # rows behind the last sequence


def test_quantised_extremes():
    x = randn((9, 1, 64), 101)
    x[0] = 0
    x[1] = 2.0 ** -130                                         # below the clamp, subnormal in bf16
    x[2] = torch.finfo(torch.bfloat16).max
    x[3, 0, 7] = math.inf
    x[4, 0, 8] = -math.inf
    x[5, 0, 9] = math.nan
    x[6] *= 2.0 ** -99
    x[7, 0, 1:] = 0
    x[8, 0, 0], x[8, 0, 1] = math.nan, math.inf
    c = Cache([9], 1, 64, 4, "e4m3", seed=102)
    args, scales = c.cuda()
    cu = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    fa.cache_write(x.cuda(), x.cuda(), *args, cu, c.seqlens.cuda(), **scales)
    code, scale = quantise(x)
    for name in ("k", "v"):
        for t in range(9):
            p, s = c.table[0, t // 4], t % 4
            got = args["kv".index(name)][p, 0, s].cpu().float()
            assert torch.equal(got, code[t, 0].float()) or (torch.isnan(got) == torch.isnan(code[t, 0].float())).all(), t
            sc = scales[name + "_scale"][p, 0, s].cpu()
            assert sc == scale[t, 0] or (torch.isnan(sc) and torch.isnan(scale[t, 0])), t
    k, v = fa.cache_read(*args, cu, c.seqlens.cuda(), 9, **scales)
    k = k.cpu().float()
    assert (k[0] == 0).all() and (k[1] == x[1].float()).logical_or(k[1].abs() <= 2.0 ** -100).all()
    assert torch.isinf(k[2]).all() or (k[2] == x[2].float()).all()
    assert k[3, 0, 7] == math.inf and k[4, 0, 8] == -math.inf and (k[3, 0, :7] == 0).all()
    assert torch.isnan(k[5]).all() and torch.isnan(k[8]).all()
    assert torch.equal(k, v.cpu().float()) or torch.isnan(v.cpu().float()[5]).all()


def test_every_code_reads_as_its_value():
    """All 256 codes through the read-back and, as values of single keys, through attention."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn)
    c = Cache([4], 1, 64, 4, "e4m3", seed=103, slack=0)
    for name in ("k", "v"):
        c.t[name + "_pages"][0, 0] = codes.view(4, 64)
        c.t[name + "_scale"][:] = 0.5
    args, scales = c.cuda()
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    k, v = fa.cache_read(*args, cu, c.seqlens.cuda(), 4, **scales)
    want = (codes.float() * 0.5).to(torch.bfloat16).view(4, 1, 64)
    fine = ~torch.isnan(want)
    assert torch.equal(k.cpu()[fine], want[fine]) and torch.equal(v.cpu()[fine], want[fine])
    assert torch.isnan(k.cpu()[~fine]).all() and int((~fine).sum()) == 2
    for n in range(1, 5):                                      # window 0: each query's output is its own value row
        L = torch.tensor([n], dtype=torch.int32, device="cuda")
        o, _ = fa.fwd_paged(torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros_like(args[0]),
                            *args[1:], L, causal=True, window=0, **scales)
        ok = fine[n - 1, 0]
        assert torch.equal(o.cpu()[0, 0, 0][ok], want[n - 1, 0][ok])
        assert torch.isnan(o.cpu()[0, 0, 0][~ok]).all()


def test_rows_without_a_place():
    """Offsets that ask for more tokens than a sequence holds, missing pages, and
    rows outside the offsets."""
    for kind in ("bf16", "e4m3"):
        c = Cache([6, 20, 3], 2, 64, 4, kind, "nhd", seed=111).fill_random(112)
        c.table[1, 2] = -1
        c.table[2, 0] = c.P
        x = randn((30, 2, 64), 113)
        cu = torch.tensor([2, 11, 27, 28], dtype=torch.int32)     # 9 rows for 6 tokens, 16 of 20, 1 of 3
        before, (args, scales) = c.cuda(), c.cuda()
        rk, rv = (torch.full((30, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        fa.cache_read(*args, cu.cuda(), c.seqlens.cuda(), 30, out=(rk, rv), **scales)
        rk = rk.cpu()
        assert (rk[:2] == 9).all() and (rk[28:] == 9).all()
        assert (rk[2:5] == 0).all()                             # positions -3 .. -1
        assert torch.equal(rk[5:11].double(), torch.from_numpy(c.rows("k", 0, torch.arange(6))).to(torch.bfloat16).double())
        assert (rk[15:19] == 0).all() and (rk[11:15] != 0).any() and (rk[27] == 0).all()   # positions 8..11 have no page
        fa.cache_write(x.cuda(), x.cuda(), *args, cu.cuda(), c.seqlens.cuda(), **scales)
        for b, n in ((0, 6), (1, 16)):
            for i in range(n):
                pos = c.lens[b] - n + i
                if b == 1 and pos // 4 == 2:
                    continue
                c.put("k", b, torch.tensor([pos]), x[cu[b + 1] - n + i][None])
                c.put("v", b, torch.tensor([pos]), x[cu[b + 1] - n + i][None])
        for got, name in zip(args[:2], ("k_pages", "v_pages")):
            assert torch.equal(got.cpu().float(), c.t[name].float()), name
        for name, got in scales.items():
            assert torch.equal(got.cpu(), c.t[name])


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_generating_tokens(kind):
    """Prompts packed through fwd_packed and into the cache, then tokens one at
    a time: each step's attention equals fwd_decode over the cache read back."""
    H, Hkv, d, page = 8, 2, 128, 16
    prompts, steps = [40, 1, 17, 130], 5
    c = Cache([n + steps for n in prompts], Hkv, d, page, kind, "nhd", seed=121)
    args, scales = c.cuda()
    B = len(prompts)
    L = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    cu = offsets(prompts).cuda()
    k, v = randn((sum(prompts), Hkv, d), 122).cuda(), randn((sum(prompts), Hkv, d), 123).cuda()
    q = randn((sum(prompts), H, d), 124).cuda()
    o, _ = fa.fwd_packed(q, k, v, [0] + list(np.cumsum(prompts)), causal=True)
    fa.cache_write(k, v, *args, cu, L, **scales)
    # the prompt's last tokens over the cache equal the packed prompt's last rows
    last = torch.stack([q[n - 1] for n in np.cumsum(prompts)])[:, :, None]
    o1, _ = fa.fwd_paged(last, *args, L, causal=True, **scales)
    if kind == "bf16":
        for b, n in enumerate(np.cumsum(prompts)):
            assert (o1[b, :, 0].float() - o[n - 1].float()).abs().max() <= 2 ** -6 * v.float().abs().max()
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    for step in range(steps):
        L += 1
        kn, vn, qn = (randn((B, h, d), 130 + 3 * step + i).cuda() for i, h in enumerate((Hkv, Hkv, H)))
        fa.cache_write(kn, vn, *args, one, L, **scales)
        o, lse = fa.fwd_paged(qn[:, :, None], *args, L, causal=True, **scales)
        lens = [n + step + 1 for n in prompts]
        dk, dv = fa.cache_read(*args, offsets(lens).cuda(), L, sum(lens), **scales)
        at = 0
        for b, n in enumerate(lens):
            kk, vv = (x[at:at + n].transpose(0, 1).contiguous()[None] for x in (dk, dv))
            want, wl = fa.fwd_decode(qn[b][None, :, None], kk, vv, causal=True)
            # bf16: the same inputs twice, each side within its rounding; e4m3: the read-back values
            # are rounded once more (half a step of K moves a score by HALF_BF16 * |q| |k| * scale)
            A = float(vv.float().abs().max())
            mag = float((kk.float().abs().amax(2).repeat_interleave(H // Hkv, 1) * qn[b].float().abs()).sum(-1).max()) / d ** 0.5
            extra = 0 if kind == "bf16" else 2 * 2 ** -8 * mag + 2 ** -8
            assert (o[b].float() - want[0].float()).abs().max() <= (4 * 2 ** -8 + extra) * A
            assert (lse[b] - wl[0]).abs().max() <= 1e-3 + (0 if kind == "bf16" else 2 ** -8 * mag)
            at += n
    assert fa.device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_captured_steps(kind):
    """A captured write + attention pair replayed while lengths and tables
    change; two graphs that use one workspace; another stream."""
    H, Hkv, d, page, B, M = 8, 2, 128, 16, 3, 40
    c = Cache([300, 20, 500], Hkv, d, page, kind, "nhd", seed=141, width=M).fill_random(142)
    args, scales = c.cuda()
    q, kn, vn = (torch.zeros((B, h, d), dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
    L = c.seqlens.cuda()
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(fa.fwd_paged_workspace_size(B, H, Hkv, 1, d), dtype=torch.uint8, device="cuda")
    outs = [(torch.empty((B, H, 1, d), dtype=torch.bfloat16, device="cuda"), torch.empty((B, H, 1), device="cuda")) for _ in range(2)]

    def step(o, lse, window):
        fa.cache_write(kn, vn, *args, one, L, **scales)
        fa.fwd_paged(q[:, :, None], *args, L, causal=True, window=window, out=o, lse=lse, workspace=ws, **scales)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*outs[0], -1)
    torch.cuda.current_stream().wait_stream(side)
    for b, n in enumerate(c.lens):                             # what that step wrote
        for name in ("k", "v"):
            c.put(name, b, torch.tensor([n - 1]), torch.zeros((1, Hkv, d), dtype=torch.bfloat16))
    graphs = []
    for (o, lse), window in zip(outs, (-1, 64)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(o, lse, window)
        graphs.append(g)
    for turn, lens in enumerate(([300, 20, 500], [1, 320, 640], [17, 1, 1], [0, 640, 2])):
        c.seqlens = torch.tensor(lens, dtype=torch.int32)
        L.copy_(c.seqlens)
        need = [-(-n // page) for n in lens]
        order = torch.randperm(c.P, generator=torch.Generator().manual_seed(turn)).int()
        table, at = torch.full((B, M), -1, dtype=torch.int32), 0
        for b, n in enumerate(need):
            n = min(n, c.P - at)                               # a pool that ran out: missing pages
            table[b, :n] = order[at:at + n]
            at += n
        c.table = table
        args[2].copy_(table)
        x = [randn(t.shape, 150 + 10 * turn + i) for i, t in enumerate((q, kn, vn))]
        for t, s in zip((q, kn, vn), x):
            t.copy_(s)
        for b, n in enumerate(lens):
            if n and 0 <= table[b, (n - 1) // page] < c.P:
                c.put("k", b, torch.tensor([n - 1]), x[1][b:b + 1])
                c.put("v", b, torch.tensor([n - 1]), x[2][b:b + 1])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (o, lse), window in zip(outs, (-1, 64)):
            want_o, want_l, tol_o, tol_l = attend(c, x[0][:, :, None], True, window)
            check("O", o, want_o, tol_o)
            check("LSE", lse, want_l, tol_l)
