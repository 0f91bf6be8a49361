"""Values, weights and scores of the paged calls at the ends of their ranges:
value scales of zero, keys of most weight whose value is zero, weights far
apart, factors that leave fp32's normal range, and the codes of extreme rows."""
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


def compare(c, q, causal=True, window=-1, **kw):
    args, scales = c.cuda()
    o, lse = fa.fwd_paged(q.cuda(), *args, c.seqlens.cuda(), causal=causal, window=window, **scales, **kw)
    torch.cuda.synchronize()
    want_o, want_l, tol_o, tol_l = attend(c, q, causal, window, kw.get("scale"))
    check("O", o, want_o, tol_o)
    check("LSE", lse, want_l, tol_l)


# sequences, kv heads, query heads a kv head, rows, head_dim: one and four kv heads a unit, 1 to 64 rows
SHAPES = [(2, 1, 1, 1, 128), (16, 4, 1, 1, 128), (16, 4, 2, 1, 64), (2, 4, 1, 1, 64), (32, 2, 3, 4, 128), (96, 4, 1, 1, 128), (2, 1, 16, 4, 64), (3, 1, 5, 4, 128)]


@pytest.mark.parametrize("B,Hkv,g,Nq,d", SHAPES)
@pytest.mark.parametrize("zeros", [16, 32, 64, 130])
def test_values_behind_scales_of_zero(B, Hkv, g, Nq, d, zeros):
    """A sequence begins with tokens whose value scale is zero (a placeholder, or
    another writer's rows of zeros) or subnormal; the tokens behind count in full."""
    for small in (0.0, 2.0 ** -140) if zeros == 64 else (0.0,):
        for lens in ([170 + 9 * b for b in range(B - 1)] + [2500], [zeros + 1 + b % 60 for b in range(B)]):
            c = Cache(lens, Hkv, d, 16, "e4m3", "nhd", seed=421).fill_random(422)
            for b in range(B):
                pid, slot = c.places(b, torch.arange(zeros))
                c.t["v_scale"][pid, :, slot] = small
            compare(c, randn((B, Hkv * g, Nq, d), 423, 2.0))
            compare(c, randn((B, Hkv * g, Nq, d), 424, 2.0), window=160)


@pytest.mark.parametrize("B,Hkv,g,Nq,d", SHAPES)
@pytest.mark.parametrize("above", [7, 14, 21])
def test_a_key_of_most_weight_without_a_value(B, Hkv, g, Nq, d, above):
    """One key's score is far above all others' and its value row is zero, with a
    scale of 2^10 or the smallest: the others make up the output."""
    n = 800
    for vscale in (None, 2.0 ** 10):
        c = Cache([n] * B, Hkv, d, 64, "e4m3", "nhd", seed=431).fill_random(432)
        q = randn((B, Hkv * g, Nq, d), 433)
        q[..., 0] = 8.0
        for b in range(B):
            at = torch.tensor([(37 * b) % 70])
            k = torch.zeros((1, Hkv, d), dtype=torch.bfloat16)
            k[..., 0] = (math.log(n) + above) * math.sqrt(d) / 8.0
            c.put("k", b, at, k)
            c.put("v", b, at, torch.zeros((1, Hkv, d), dtype=torch.bfloat16))
            if vscale is not None:
                pid, slot = c.places(b, at)
                c.t["v_scale"][pid, :, slot] = vscale
        compare(c, q)


@pytest.mark.parametrize("B,Hkv,g,Nq,d", SHAPES)
def test_weights_far_apart(B, Hkv, g, Nq, d):
    """Scores spread over a hundred and more, values larger the smaller their weight."""
    lens = [90 + 7 * b for b in range(B)]
    c = Cache(lens, Hkv, d, 16, "e4m3", "nhd", seed=441).fill_random(442)
    q = randn((B, Hkv * g, Nq, d), 443)
    q[..., 0] = 8.0
    for b, n in enumerate(lens):
        for j in range(n):
            s = (j * 29) % 97                                  # the score, about
            k = randn((1, Hkv, d), 444 + j, 0.1)
            k[..., 0] = s * math.sqrt(d) / 8.0
            c.put("k", b, torch.tensor([j]), k)
            c.put("v", b, torch.tensor([j]), randn((1, Hkv, d), 644 + j, 2.0 ** min(127, 100 - s)) if s % 3 else
                  torch.zeros((1, Hkv, d), dtype=torch.bfloat16))
    compare(c, q)
    compare(c, q, window=20)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [1e-44, 1e-30, 1e-13, 2e38])
def test_rows_of_zeros_under_any_scale(kind, scale):
    """Rows without a score of their own: the mean of the values that the mask leaves."""
    for B, Hkv, g, Nq, d in SHAPES[:5]:
        lens = [20 + 11 * b for b in range(B - 1)] + [700]
        c = Cache(lens, Hkv, d, 16, kind, "nhd", seed=451).fill_random(452)
        q = torch.zeros((B, Hkv * g, Nq, d), dtype=torch.bfloat16)
        compare(c, q, scale=scale)
        compare(c, q, causal=False, window=9, scale=scale)
        if scale < 1:
            q[..., 1] = 2.0 ** -110
            compare(c, q, window=9, scale=scale)
        else:                                                  # keys of zeros, queries of any size
            c.t["k_pages"].zero_()
            q[..., 2:] = 2.0 ** 100
            compare(c, q, window=9, scale=scale)


def test_codes_and_values_of_extreme_rows():
    """Every code, scale and value read back is the definition's in fp32, NaN where it is NaN."""
    top = torch.finfo(torch.bfloat16).max
    x = {"k": randn((10, 2, 64), 461), "v": randn((10, 2, 64), 462)}
    for t in x.values():
        t[0] = 0
        t[1] = 2.0 ** -130                                     # below the clamp, subnormal in bf16
        t[2] = top
        t[3, 0, 7] = math.inf
        t[4, 1, 8] = -math.inf
        t[5, 0, 9] = math.nan
        t[6] *= 2.0 ** -99
        t[7, 0, 1:] = 0
        t[8, 0, 0], t[8, 0, 1] = math.nan, math.inf
        t[9, :, :32], t[9, :, 32:] = top, -2.0 ** 120
    c = Cache([10], 2, 64, 4, "e4m3", seed=463)
    (k, v, table), scales = c.cuda()
    cu, L = torch.tensor([0, 10], dtype=torch.int32, device="cuda"), c.seqlens.cuda()
    fa.cache_write(x["k"].cuda(), x["v"].cuda(), k, v, table, cu, L, **scales)
    rk, rv = fa.cache_read(k, v, table, cu, L, 10, **scales)
    pid, slot = c.places(0, torch.arange(10))
    for name, pages, back in (("k", k, rk), ("v", v, rv)):
        code, scale = quantise(x[name])
        got = pages.cpu().view(torch.uint8)[pid, :, slot].view(torch.float8_e4m3fn).float()
        torch.testing.assert_close(got, code.float(), rtol=0, atol=0, equal_nan=True)
        torch.testing.assert_close(scales[name + "_scale"].cpu()[pid, :, slot], scale, rtol=0, atol=0, equal_nan=True)
        want = (code.float() * scale[..., None]).to(torch.bfloat16)
        torch.testing.assert_close(back.cpu(), want, rtol=0, atol=0, equal_nan=True)
        assert int(torch.isnan(want).sum()) == 2 * 64 and torch.isinf(want).any()


def test_windows_wider_than_any_cache():
    """Half-widths beyond 32 bits are wide windows, not their low 32 bits; numbers below -1 are refused."""
    c = Cache([90, 300], 2, 64, 16, "bf16", "nhd", seed=471).fill_random(472)
    args, _ = c.cuda()
    L, q = c.seqlens.cuda(), randn((2, 4, 1, 64), 473).cuda()
    want = fa.fwd_paged(q, *args, L, causal=True)
    for window in (300, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 10 ** 12, 2 ** 64):
        o, lse = fa.fwd_paged(q, *args, L, causal=True, window=window)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), window
    for window in (-2, -2 ** 31, -2 ** 32 - 1, -2 ** 64):
        with pytest.raises(fa.FAError):
            fa.fwd_paged(q, *args, L, causal=True, window=window)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_chunk_of_a_prompt(kind):
    """Hundreds of new tokens over a cache: many blocks of rows, more units of a sequence than CTAs."""
    c = Cache([700, 130, 0], 8, 64, 16, kind, "nhd", seed=481).fill_random(482)
    compare(c, randn((3, 16, 260, 64), 483, 2.0))
    compare(c, randn((3, 16, 260, 64), 484, 2.0), window=40)
