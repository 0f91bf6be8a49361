"""What the paged calls' warps and kernels hand to one another: states joined at
the end of short units, and tensors that the kernel before still writes."""
import pytest
import torch

import exact_io_aware_online_b200 as fa

from paged_ref import Cache, attend, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_online_b200 import _build
    _build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def randn(shape, seed, spread=1.0):
    return (torch.randn(shape, generator=torch.Generator("cpu").manual_seed(seed)) * spread).to(torch.bfloat16)


@pytest.mark.parametrize("kind,d,Hkv,g,Nq", [("bf16", 128, 2, 1, 1), ("bf16", 128, 1, 2, 2), ("bf16", 64, 1, 1, 1), ("bf16", 64, 1, 12, 1),
                                             ("e4m3", 128, 1, 1, 1), ("e4m3", 64, 1, 12, 1)])
def test_states_joined_unit_after_unit(kind, d, Hkv, g, Nq):
    """Units of one tile, one behind the other, whose keys are shared by four or
    two warps: many keys in one unit, in the next so few that most warps have none
    and come to the unit's end at once."""
    B = 2400
    gen = torch.Generator().manual_seed(401)
    lens = [int(torch.randint(*((50, 64) if b % 2 else (1, 8)), (1,), generator=gen)) for b in range(B)]
    c = Cache(lens, Hkv, d, 16, kind, "nhd", seed=402).fill_random(403)
    q = randn((B, Hkv * g, Nq, d), 404, 2.0)
    (k, v, table), scales = c.cuda()
    L, qd = c.seqlens.cuda(), q.cuda()
    first = fa.fwd_paged(qd, k, v, table, L, causal=True, **scales)
    want_o, want_l, tol_o, tol_l = attend(c, q, True, -1)
    check("O", first[0], want_o, tol_o)
    check("LSE", first[1], want_l, tol_l)
    for _ in range(20):
        o, lse = fa.fwd_paged(qd, k, v, table, L, causal=True, **scales)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_tensors_that_the_call_before_wrote(kind):
    """Tokens go from one cache into another and back through the same buffers,
    and queries into the buffer that the attention before wrote, without a pause."""
    n, Hkv, d = 700, 4, 128
    one, two = (Cache([n], Hkv, d, 16, kind, "nhd", seed=411 + i) for i in range(2))
    one.fill_random(413)
    a, sa = one.cuda()
    b, sb = two.cuda()
    L, cu = one.seqlens.cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    k, v = (torch.zeros((n, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = randn((1, 8, 1, d), 414, 2.0).cuda()
    bufs = [torch.zeros_like(q) for _ in range(3)]
    fa.cache_read(*a, cu, L, n, out=(k, v), **sa)
    fa.cache_write(k, v, *b, cu, L, **sb)
    torch.cuda.synchronize()
    want = [q]
    for _ in range(2):
        want.append(fa.fwd_paged(want[-1], *b, L, causal=True, **sb)[0])
        torch.cuda.synchronize()
    first = k.clone(), v.clone()
    for _ in range(30):
        for t in (k, v, *b[:2], *bufs):
            t.zero_()
        bufs[0].copy_(q)
        fa.cache_read(*a, cu, L, n, out=(k, v), **sa)
        fa.cache_write(k, v, *b, cu, L, **sb)
        fa.fwd_paged(bufs[0], *b, L, causal=True, out=bufs[1], **sb)
        fa.fwd_paged(bufs[1], *b, L, causal=True, out=bufs[2], **sb)
        fa.cache_read(*b, cu, L, n, out=(k, v), **sb)
        torch.cuda.synchronize()
        assert torch.equal(bufs[1], want[1]) and torch.equal(bufs[2], want[2])
        if kind == "bf16":                                     # codes of codes: a second rounding
            assert torch.equal(k, first[0]) and torch.equal(v, first[1])
