"""Workloads of the paged key/value cache: writing tokens into it, reading it back, and attention over it.

Each case is one call of a serving program.  With `own` false `run` computes the operators from
elementary torch operations in fp32 (rounded once at the end); with `own` true it calls the
framework.  Sizes: 32 query heads on 8 kv heads at d = 128 and 16 heads at d = 64 are the
framework's own workloads', as is the 32768-token cache of 8 sequences; the rest are generic.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_LO = 2.0 ** -100                 # a row's largest magnitude is clamped to [2^-100, FLT_MAX]
AMAX_HI = torch.finfo(torch.float32).max


def _att(name, B, H, Hkv, d, lo, hi, page, kind, layout, Nq=1, window=-1):
    return {"name": name, "op": "attend", "B": B, "H": H, "Hkv": Hkv, "d": d, "lo": lo, "hi": hi, "page": page,
            "kind": kind, "layout": layout, "Nq": Nq, "window": window, "lens": 1}


def _mov(name, op, B, Hkv, d, lo, hi, page, kind, layout, new=0):
    return {"name": name, "op": op, "B": B, "Hkv": Hkv, "d": d, "lo": lo, "hi": hi, "page": page, "kind": kind,
            "layout": layout, "new": new, "lens": 1}


def listed():
    return [
        # one user, the next token after a short prompt: latency counts
        _att("token_b1_n1000_bf16", 1, 32, 8, 128, 1000, 1000, 16, "bf16", "hnd"),
        # the framework's long decode: 8 sequences of 32768 tokens
        _att("token_b8_n32768_bf16", 8, 32, 8, 128, 32768, 32768, 128, "bf16", "hnd"),
        # a serving batch with lengths all over the range, tokens outer in a page
        _att("ragged_b64_bf16", 64, 32, 8, 128, 16, 16384, 16, "bf16", "nhd"),
        # the same kind of batch on the quantised cache, eight query heads a kv head
        _att("ragged_b128_e4m3", 128, 64, 8, 128, 64, 8192, 64, "e4m3", "nhd"),
        # four drafted tokens a sequence, checked at once (causal among themselves)
        _att("draft4_b16_e4m3", 16, 32, 8, 128, 2000, 12000, 32, "e4m3", "hnd", Nq=4),
        # many short chats on a model with a sliding window and one query head a kv head
        _att("window_b256_d64_bf16", 256, 16, 16, 64, 1, 4096, 16, "bf16", "nhd", window=255),
        # the step's new tokens go into the cache: one a sequence
        _mov("write_token_b64_e4m3", "write", 64, 8, 128, 16, 16384, 16, "e4m3", "nhd", new=1),
        # prompts of a batch, K and V slices of one fused projection buffer
        _mov("write_prompts_b16_bf16", "write", 16, 8, 128, 30, 4000, 16, "bf16", "hnd"),
        # a large prefill, quantised
        _mov("write_prompts_b8_e4m3", "write", 8, 8, 128, 16384, 16384, 64, "e4m3", "nhd"),
        # one cached prompt back as dense tensors, for a following chunk
        _mov("read_b1_n1000_bf16", "read", 1, 8, 128, 1000, 1000, 16, "bf16", "hnd"),
        # a whole batch's quantised cache back as packed sequences
        _mov("read_b32_e4m3", "read", 32, 8, 128, 100, 16384, 32, "e4m3", "nhd"),
        # small heads, many short sequences
        _mov("read_b256_d64_bf16", "read", 256, 16, 64, 1, 1000, 16, "bf16", "hnd"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    kind = rng.choice(["bf16", "e4m3"])
    page = rng.choice([8, 16, 32, 48, 64, 128])
    layout = rng.choice(["hnd", "nhd"])
    op = rng.choice(["attend", "attend", "write", "read"])
    B = _log(rng, 1, 256)
    es = 2 if kind == "bf16" else 1
    room = 1.0e9 / (2 * d * Hkv * es) if op == "attend" else 4.0e8 / (6 * d * Hkv)  # tokens within the largest case
    hi = min(_log(rng, 4, 32768), max(1, int(room // B)))
    lo = max(1, hi - rng.randrange(hi)) if rng.random() < 0.7 else hi
    c = {"op": op, "B": B, "Hkv": Hkv, "d": d, "lo": lo, "hi": hi, "page": page, "kind": kind, "layout": layout,
         "lens": rng.randrange(1 << 20)}
    if op == "attend":
        c["H"] = Hkv * rng.choice([1, 2, 3, 4, 8, 16] if Hkv < 16 else [1, 2, 4])
        c["Nq"] = rng.choice([1, 1, 1, 2, 4])
        c["window"] = rng.choice([-1, -1, _log(rng, 16, 4096)])
    else:
        c["new"] = rng.choice([0, 1, 3]) if op == "write" else 0
    return c


def _lengths(case):
    """Tokens of each sequence (log-uniform over [lo, hi]), a property of the case."""
    lo, hi = case["lo"], case["hi"]
    g = torch.Generator("cpu").manual_seed(case["lens"])
    u = torch.rand(case["B"], generator=g, dtype=torch.float64)
    n = torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo))).round().long().clamp(lo, hi)
    n[0] = hi
    return n


def _new(case, n):
    """Tokens of each sequence that the call moves: the newest `new`, or all of them."""
    return n.clamp(max=case["new"]) if case["new"] else n


def _quantise(x):
    """Codes (e4m3) and scales of rows x [..., d], in fp32."""
    x = x.float()
    a = x.abs().amax(-1).clamp(AMAX_LO, AMAX_HI)
    up = torch.full_like(a, E4M3_MAX) / a           # a true division: number / tensor multiplies by a reciprocal
    return (x * up[..., None]).to(torch.float8_e4m3fn), a / E4M3_MAX


def _pages(shape, layout, make):
    """A [P, Hkv, page, d] tensor, tokens outside heads in memory where layout is "nhd"."""
    P, Hkv, page, d = shape
    return make((P, page, Hkv, d)).transpose(1, 2) if layout == "nhd" else make(shape)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    n = _lengths(case)
    per = (n + page - 1) // page
    width, used = int(per.max()), int(per.sum())
    P = used + 3                                    # a pool with a few free pages
    order = torch.randperm(P, generator=g, device="cuda")[:used].int()
    valid = torch.arange(width, device="cuda")[None, :] < per.cuda()[:, None]
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[valid] = order

    def randn(shape, spread=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * spread

    s = {"case": case, "table": table, "seqlens": n.int().cuda()}
    names = ("k", "v")
    for name in names:
        s[name + "_scale"] = None
        if case["kind"] == "bf16":
            s[name + "_pages"] = _pages((P, Hkv, page, d), case["layout"], randn)
            continue
        full = torch.empty((P, page, Hkv, d) if case["layout"] == "nhd" else (P, Hkv, page, d), dtype=torch.float8_e4m3fn,
                           device="cuda")
        scale = torch.empty(full.shape[:3], device="cuda")
        for at in range(0, P, 4096):                # in slices: a cache is large
            x = randn((min(4096, P - at), *full.shape[1:]))
            full[at:at + 4096], scale[at:at + 4096] = _quantise(x)
        nhd = case["layout"] == "nhd"
        s[name + "_pages"] = full.transpose(1, 2) if nhd else full
        s[name + "_scale"] = scale.transpose(1, 2) if nhd else scale
    if case["op"] == "attend":
        s["q"] = randn((B, case["H"], case["Nq"], d))
        return s
    cnt = _new(case, n)
    s["cu"] = torch.cat([torch.zeros(1, dtype=torch.long), cnt.cumsum(0)]).int().cuda()
    s["T"] = int(cnt.sum())
    if case["op"] == "write":                       # K and V slices of a fused projection's output
        qkv = randn((s["T"], 4 * Hkv, d))
        s["k"], s["v"] = qkv[:, 2 * Hkv:3 * Hkv], qkv[:, 3 * Hkv:]
    return s


def _gather(pages, scale, page_id, slot):
    """fp32 rows [..., Hkv, d] of the slots (page_id, slot)."""
    if scale is None:
        return pages[page_id, :, slot].float()
    x = pages.view(torch.uint8)[page_id, :, slot].view(torch.float8_e4m3fn).float()
    return x * scale[page_id, :, slot][..., None]


def _places(s):
    """Page and slot of every moved token: those of sequence b are the newest of its seqlens[b]."""
    cu, page = s["cu"].long(), s["case"]["page"]
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = s["seqlens"].long()[b] - cu[b + 1] + t
    return s["table"][b, pos // page].long(), pos % page


def _attend(s):
    case = s["case"]
    B, H, Hkv, d, Nq, w, page = (case[x] for x in ("B", "H", "Hkv", "d", "Nq", "window", "page"))
    L = s["seqlens"].long()
    pos = torch.arange(s["table"].shape[1] * page, device="cuda")
    pid = s["table"].long().clamp(min=0)[:, pos // page]
    p = (L - Nq)[:, None] + torch.arange(Nq, device="cuda")[None, :]
    keep = (pos[None, None, :] <= p[:, :, None]) & (pos[None, None, :] < L[:, None, None]) & (p[:, :, None] >= 0)
    if w >= 0:
        keep &= pos[None, None, :] >= p[:, :, None] - w
    K = _gather(s["k_pages"], s["k_scale"], pid, pos % page)            # [B, N, Hkv, d]
    q = s["q"].float().view(B, Hkv, H // Hkv * Nq, d)
    S = torch.matmul(q, K.permute(0, 2, 3, 1)) / math.sqrt(d)
    del K
    S = S.view(B, Hkv, H // Hkv, Nq, -1).masked_fill(~keep[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(S - m0)
    l = e.sum(-1, keepdim=True)
    V = _gather(s["v_pages"], s["v_scale"], pid, pos % page)
    O = torch.matmul(e.view(B, Hkv, H // Hkv * Nq, -1), V.permute(0, 2, 1, 3)).view(B, Hkv, H // Hkv, Nq, d)
    O = torch.where(l > 0, O / l, torch.zeros_like(O))
    return {"o": O.view(B, H, Nq, d).bfloat16(), "lse": (m + torch.log(l)).view(B, H, Nq)}


def _write(s):
    pid, slot = _places(s)
    for name in ("k", "v"):
        x, pages = s[name], s[name + "_pages"]
        if s[name + "_scale"] is None:
            pages[pid, :, slot] = x
        else:
            code, scale = _quantise(x)
            pages.view(torch.uint8)[pid, :, slot] = code.view(torch.uint8)
            s[name + "_scale"][pid, :, slot] = scale


def run(s):
    op = s["case"]["op"]
    if own:
        import exact_io_aware_online_b200 as fa
        cache = (s["k_pages"], s["v_pages"], s["table"])
        scales = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if op == "attend":
        if own:
            o, lse = fa.fwd_paged(s["q"], *cache, s["seqlens"], causal=True, window=s["case"]["window"], **scales)
            return {"o": o, "lse": lse}
        return _attend(s)
    if op == "read":
        if own:
            k, v = fa.cache_read(*cache, s["cu"], s["seqlens"], s["T"], **scales)
        else:
            pid, slot = _places(s)
            k = _gather(s["k_pages"], s["k_scale"], pid, slot).bfloat16()
            v = _gather(s["v_pages"], s["v_scale"], pid, slot).bfloat16()
        return {"k": k, "v": v}
    if own:
        fa.cache_write(s["k"], s["v"], *cache, s["cu"], s["seqlens"], **scales)
    else:
        _write(s)
    out = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["k_scale"] is not None:
        out |= {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return out


def work(case):
    n, d, Hkv, B = _lengths(case), case["d"], case["Hkv"], case["B"]
    row = 2 * d if case["kind"] == "bf16" else d + 4         # bytes of a cached row of one kv head
    if case["op"] == "attend":
        H, Nq, w = case["H"], case["Nq"], case["window"]
        first = (n - Nq).clamp(min=0)                         # position of the first query that is a token
        seen = n if w < 0 else n - (first - w).clamp(min=0)
        p = n[:, None] - Nq + torch.arange(Nq)[None, :]
        pairs = (p + 1).clamp(min=0) if w < 0 else (p + 1).clamp(min=0, max=w + 1)
        per = (seen + case["page"] - 1) // case["page"]
        return {"bytes": int(seen.sum()) * Hkv * 2 * row + B * H * Nq * (4 * d + 4) + 4 * int(per.sum()) + 4 * B,
                "flops": 4 * d * H * int(pairs.sum())}
    T = int(_new(case, n).sum())
    return {"bytes": T * Hkv * 2 * (2 * d + row) + 8 * B, "flops": 2 * T * Hkv * 2 * d if case["kind"] == "e4m3" else 0}


def exact(case, seed):
    s = prepare(case, seed)
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    table, L = s["table"].long().cpu(), s["seqlens"].tolist()

    def rows(name, b, lo, hi):
        """Positions [lo, hi) of sequence b in 64 bits: [Hkv, hi - lo, d]."""
        at = torch.arange(lo, hi)
        pid, slot = table[b, at // page].cuda(), (at % page).cuda()
        x = s[name + "_pages"]
        x = x[pid, :, slot].double() if x.dtype == torch.bfloat16 else x.view(torch.uint8)[pid, :, slot].view(x.dtype).double()
        if s[name + "_scale"] is not None:
            x = x * s[name + "_scale"][pid, :, slot].double()[..., None]
        return x.transpose(0, 1)

    if case["op"] == "attend":
        H, Nq, w = case["H"], case["Nq"], case["window"]
        o = torch.zeros((B, H, Nq, d), dtype=torch.float64, device="cuda")
        lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            for i in range(Nq):
                p = L[b] - Nq + i
                if p < 0:
                    continue
                lo = 0 if w < 0 else max(0, p - w)
                K, V = rows("k", b, lo, p + 1), rows("v", b, lo, p + 1)
                q = s["q"][b, :, i].double().view(Hkv, H // Hkv, d)
                S = torch.einsum("hgd,hnd->hgn", q, K) / math.sqrt(d)
                lse[b, :, i] = torch.logsumexp(S, -1).reshape(H)
                o[b, :, i] = torch.einsum("hgn,hnd->hgd", torch.softmax(S, -1), V).reshape(H, d)
        return {"o": o, "lse": lse}
    cu = s["cu"].tolist()
    if case["op"] == "read":
        out = {}
        for name in ("k", "v"):
            out[name] = torch.cat([rows(name, b, L[b] - (cu[b + 1] - cu[b]), L[b]).transpose(0, 1) for b in range(B)])
        return out
    out = {}
    for name in ("k", "v"):
        pages, scale = s[name + "_pages"].double(), s[name + "_scale"]
        scale = None if scale is None else scale.double()
        for b in range(B):
            at = torch.arange(L[b] - (cu[b + 1] - cu[b]), L[b])
            pid, slot = table[b, at // page].cuda(), (at % page).cuda()
            x = s[name][cu[b]:cu[b + 1]].double()
            if scale is not None:
                a = x.abs().amax(-1).clamp(AMAX_LO, AMAX_HI)
                scale[pid, :, slot] = a / E4M3_MAX
                x = x * (E4M3_MAX / a)[..., None]     # before its rounding to a code
            pages[pid, :, slot] = x
        out[name + "_pages"] = pages
        if scale is not None:
            out[name + "_scale"] = scale
    return out
