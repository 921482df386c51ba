"""The measured cases of the serving-step operators: planning pages on the GPU,
rotary positions with several axes, the 8-bit paged cache's write side and the
attention that reads it, each with its plain form in elementary torch
operations and its definition in 64 bits.
"""
import math

import torch

own = False


def _ops():
    from exact_attention_94_gb300 import ops
    return ops


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a busy server: every request gets one token
        dict(name="plan decode step", op="plan", B=256, new_lo=1, new_hi=1, ctx_hi=8192, P=16, pad=0),
        # a mixed step: prompts of very different lengths beside requests that continue, capacity padded
        dict(name="plan prompts", op="plan", B=61, new_lo=1, new_hi=4095, ctx_hi=777, P=16, pad=1000),
        # the rotary of one decode step
        dict(name="rope decode step", op="rope", T=64, Hq=32, Hkv=8, d=128, n_axes=1, per_axis=0, neighbours=0, bwd=0),
        # a prompt with images: text and patches, three axes over one ladder of frequencies
        dict(name="rope image prompt", op="rope", T=16384, Hq=32, Hkv=8, d=128, n_axes=3, per_axis=0, neighbours=0, bwd=0),
        # training on video patches: the gradients, a ladder for each axis, odd length
        dict(name="rope video gradient", op="rope", T=12289, Hq=16, Hkv=16, d=64, n_axes=3, per_axis=1, neighbours=1, bwd=1),
        # the cache write of one decode step, most pages partly filled
        dict(name="append decode step", op="append", B=64, new=1, ctx_hi=4096, P=16, Hkv=8, d=128),
        # the cache write of long prompts, odd lengths
        dict(name="append prompts", op="append", B=9, new=2047, ctx_hi=100, P=32, Hkv=8, d=128),
        # a single short request: latency
        dict(name="decode one request", op="decode", B=1, Nq=1, Hq=32, Hkv=8, d=128, L_lo=777, L_hi=777, P=16, window=-1),
        # a full batch over long ragged caches
        dict(name="decode long batch", op="decode", B=64, Nq=1, Hq=64, Hkv=8, d=128, L_lo=16385, L_hi=32768, P=16, window=-1),
        # one K/V head for each query head
        dict(name="decode multi-head", op="decode", B=8, Nq=1, Hq=32, Hkv=32, d=128, L_lo=1000, L_hi=8192, P=64, window=-1),
        # drafts verified by the target model: four tokens a request
        dict(name="decode drafts", op="decode", B=16, Nq=4, Hq=64, Hkv=8, d=128, L_lo=100, L_hi=16384, P=32, window=-1),
        # sliding-window layers, narrow heads
        dict(name="decode window", op="decode", B=32, Nq=1, Hq=16, Hkv=4, d=64, L_lo=1, L_hi=32768, P=16, window=4095),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "decode", "decode"])
    P = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 2048)
        hi = _log(rng, 1, max(1, min(8192, 262144 // B)))
        return dict(op=op, B=B, new_lo=rng.choice([0, 1, hi]), new_hi=hi, ctx_hi=_log(rng, 1, 8192), P=P,
                    pad=rng.choice([0, 1, 77, 1000]))
    if op == "rope":
        Hkv = rng.choice([1, 2, 4, 8, 16])
        Hq = Hkv * rng.choice([1, 2, 4, 7])
        d = rng.choice([64, 128])
        T = _log(rng, 1, max(1, min(65536, 80000000 // (d * (Hq + Hkv)))))
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, d=d, n_axes=rng.choice([1, 2, 3]), per_axis=rng.choice([0, 1]),
                    neighbours=rng.choice([0, 1]), bwd=rng.choice([0, 1]))
    if op == "append":
        Hkv, d = rng.choice([1, 2, 4, 8, 32]), rng.choice([64, 128])
        n = _log(rng, 1, max(1, min(32768, 20000000 // (Hkv * d))))
        B = min(n, _log(rng, 1, 512))
        return dict(op=op, B=B, new=max(1, n // B), ctx_hi=_log(rng, 1, 2048), P=P, Hkv=Hkv, d=d)
    Hkv, d = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 128])
    B = _log(rng, 1, 96)
    Nq, Hq = rng.choice([1, 1, 1, 2, 3, 8]), Hkv * rng.choice([1, 2, 4, 5, 8])
    L = _log(rng, 1, max(1, min(65536, 1000000000 // (B * Hkv * d), 12000000000 // (B * Hq * Nq * d))))
    return dict(op=op, B=B, Nq=Nq, Hq=Hq, Hkv=Hkv, d=d,
                L_lo=rng.choice([0, 1, L // 2, L]), L_hi=L, P=P, window=rng.choice([-1, -1, 0, L // 3, 1023]))


def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spread: their sum does not depend on the seed, their order does."""
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _shuffled(values, g):
    t = torch.tensor(values, dtype=torch.int32, device="cuda")
    return t[torch.randperm(len(values), generator=g, device="cuda")].contiguous()


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s; 0 for 0."""
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m == 0.5, e - 1, e).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _encode(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _pages(num_pages, Hkv, P, d, g, keys):
    """A cache of num_pages pages as an earlier step has left it: codes and a scale for each page and head.
    Keys have a few loud channels, as trained models' keys do."""
    codes = torch.empty((num_pages, Hkv, P, d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((num_pages, Hkv), dtype=torch.float32, device="cuda")
    loud = torch.ones(d, device="cuda")
    if keys:
        loud[torch.randperm(d, generator=g, device="cuda")[: d // 16]] = 4.0
    step = max(1, (1 << 27) // (Hkv * P * d))
    for a in range(0, num_pages, step):
        b = min(num_pages, a + step)
        x = torch.randn((b - a, Hkv, P, d), generator=g, device="cuda") * loud
        s = _pow2_scale(x.abs().amax(dim=(2, 3)))
        codes[a:b] = _encode(x / s[:, :, None, None])
        scales[a:b] = s
    return codes, scales


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    return {"plan": _prepare_plan, "rope": _prepare_rope, "append": _prepare_append,
            "decode": _prepare_decode}[c["op"]](c, g)


def _prepare_plan(c, g):
    B, P = c["B"], c["P"]
    new = _spread(c["new_lo"], c["new_hi"], B)
    ctx = _spread(0, c["ctx_hi"], B)
    max_blocks = -(-(c["ctx_hi"] + c["new_hi"]) // P)
    need = sum(-(-(a + n) // P) for a, n in zip(ctx, [c["new_hi"]] * B))
    held = [-(-a // P) for a in ctx]
    num_pages = need + 7
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    ctx_lens = _shuffled(ctx, g)
    blocks = (ctx_lens + P - 1) // P
    first = torch.cumsum(blocks, 0) - blocks
    cols = torch.arange(max_blocks, device="cuda")[None]
    table = torch.where(cols < blocks[:, None], order[(first[:, None] + cols).clamp(max=num_pages - 1)], 0).to(torch.int32)
    free = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    left = num_pages - sum(held)
    free[:left] = order[sum(held):]
    return dict(case=c, ctx_lens=ctx_lens, new_lens=_shuffled(new, g), free_pages=free,
                free_count=torch.tensor([left], dtype=torch.int32, device="cuda"), table=table.contiguous(),
                max_tokens=sum(new) + c["pad"])


def _frequencies(c):
    """(axis of each pair, frequency of each pair) as plain lists."""
    half, A = c["d"] // 2, c["n_axes"]
    sizes = [half] if A == 1 else [half // 2, half - half // 2] if A == 2 else [half // 4, half // 8 * 3, half - half // 4 - half // 8 * 3]
    axis = [a for a in range(A) for _ in range(sizes[a])]
    if c["per_axis"]:
        freq = [10000.0 ** (-j / sizes[a]) for a in range(A) for j in range(sizes[a])]
    else:
        freq = [1000000.0 ** (-i / half) for i in range(half)]
    return axis, freq


def _prepare_rope(c, g):
    T, Hq, Hkv, d, A = c["T"], c["Hq"], c["Hkv"], c["d"], c["n_axes"]
    # q, k and v come out of one projection: rows of q and k are slices of its rows
    qkv = torch.randn((T, (Hq + 2 * Hkv) * d), generator=g, device="cuda").to(torch.bfloat16)
    q = qkv[:, : Hq * d].unflatten(1, (Hq, d))
    k = qkv[:, Hq * d: (Hq + Hkv) * d].unflatten(1, (Hkv, d))
    start = torch.randint(0, 100000, (1,), generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    text = T // 4  # text first, then patches of 24 x 32 frames
    patch = (t - text).clamp(min=0)
    grid = torch.stack([patch // 768, patch // 32 % 24, patch % 32])[-A:] + text if A > 1 else t[None]
    pos = torch.where(t < text, t[None].expand(A, T), grid) + start
    axis, freq = _frequencies(c)
    s = dict(case=c, q=q, k=k, positions=pos.to(torch.int32).contiguous(),
             axis=torch.tensor(axis, device="cuda"), freq=torch.tensor(freq, dtype=torch.float64, device="cuda"))
    if own:
        s["plan"] = _ops().RopePlan(d, axis, freq, neighbours=bool(c["neighbours"]))
    return s


def _prepare_append(c, g):
    B, P, Hkv, d, n = c["B"], c["P"], c["Hkv"], c["d"], c["new"]
    ctx = _shuffled(_spread(0, c["ctx_hi"], B), g)
    per = n // P + 2  # pages a request can touch
    num_pages = B * per + 3
    order = torch.randperm(num_pages, generator=g, device="cuda")
    t = torch.arange(B * n, device="cuda")
    b, pos = t // n, ctx[t // n] + t % n
    page = order[b * per + pos // P - ctx[b] // P]
    kc, ks = _pages(num_pages, Hkv, P, d, g, True)
    vc, vs = _pages(num_pages, Hkv, P, d, g, False)
    # slices of one projection's rows; one token in eight is louder than what its page holds
    kv = torch.randn((B * n, 2 * Hkv * d), generator=g, device="cuda")
    kv = kv * torch.where(torch.rand((B * n, 1), generator=g, device="cuda") < 0.125, 4.0, 1.0)
    kv = kv.to(torch.bfloat16)
    return dict(case=c, k_new=kv[:, : Hkv * d].unflatten(1, (Hkv, d)), v_new=kv[:, Hkv * d:].unflatten(1, (Hkv, d)),
                k_codes=kc, v_codes=vc, k_scale=ks, v_scale=vs, page=page.to(torch.int32).contiguous(),
                slot=(pos % P).to(torch.int32).contiguous())


def _prepare_decode(c, g):
    B, P, Hkv, Hq, d = c["B"], c["P"], c["Hkv"], c["Hq"], c["d"]
    lens = _spread(c["L_lo"], c["L_hi"], B)
    seq_lens = _shuffled(lens, g)
    blocks = (seq_lens + P - 1) // P
    max_blocks = max(1, -(-c["L_hi"] // P))
    num_pages = sum(-(-n // P) for n in lens) + 3
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(blocks, 0) - blocks
    cols = torch.arange(max_blocks, device="cuda")[None]
    table = torch.where(cols < blocks[:, None], order[(first[:, None] + cols).clamp(max=num_pages - 1)], 0).to(torch.int32)
    kc, ks = _pages(num_pages, Hkv, P, d, g, True)
    vc, vs = _pages(num_pages, Hkv, P, d, g, False)
    q = torch.randn((B, c["Nq"], Hq, d), generator=g, device="cuda").to(torch.bfloat16)
    return dict(case=c, q=q, k_codes=kc, v_codes=vc, k_scale=ks, v_scale=vs, table=table.contiguous(), seq_lens=seq_lens)


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    return {"plan": _run_plan, "rope": _run_rope, "append": _run_append, "decode": _run_decode}[c["op"]](s, c)


def _run_plan(s, c):
    if own:
        p = _ops().page_plan(s["ctx_lens"], s["new_lens"], s["free_pages"], s["free_count"], s["table"], c["P"], s["max_tokens"])
        return p.seq_lens, p.cu_new, p.page, p.slot, p.position, p.free_count, s["table"]
    ctx, new, table, P = s["ctx_lens"], s["new_lens"], s["table"], c["P"]
    B, max_blocks = table.shape
    seq = ctx + new
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.cumsum(new, 0)
    first = (ctx + P - 1) // P
    end = (seq + P - 1) // P
    need = end - first
    base = torch.cumsum(need, 0) - need
    cols = torch.arange(max_blocks, device="cuda")[None]
    at = s["free_count"] - 1 - (base[:, None] + cols - first[:, None])
    fresh = (cols >= first[:, None]) & (cols < end[:, None])
    table.copy_(torch.where(fresh, s["free_pages"][at.clamp(0, s["free_pages"].numel() - 1)], table))
    rows = torch.arange(s["max_tokens"], dtype=torch.int32, device="cuda")
    b = torch.searchsorted(cu[1:], rows, right=True).clamp(max=B - 1)
    real = rows < cu[-1]
    pos = torch.where(real, ctx[b] + rows - cu[b], 0)
    page = torch.where(real, table[b, pos // P], -1)
    slot = torch.where(real, pos % P, -1)
    return seq, cu, page, slot, pos, s["free_count"] - need.sum().to(torch.int32), table


def _rotate(x, ca, sa, neighbours):
    """x [T, H, d] in 32 or 64 bits; ca, sa [T, 1, d / 2]."""
    if neighbours:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * ca - b * sa, a * sa + b * ca], dim=-1).flatten(-2)
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * ca - b * sa, a * sa + b * ca], dim=-1)


def _run_rope(s, c):
    if own:
        f = _ops().rope_axes_bwd if c["bwd"] else _ops().rope_axes
        return f(s["q"], s["k"], s["positions"], s["plan"])
    angle = s["positions"].t()[:, s["axis"]].double() * s["freq"]
    ca, sa = angle.cos().float()[:, None], angle.sin().float()[:, None]
    sa = -sa if c["bwd"] else sa
    return tuple(_rotate(x.float(), ca, sa, c["neighbours"]).to(torch.bfloat16) for x in (s["q"], s["k"]))


def _append_one(x, codes, scales, page, slot):
    num_pages, Hkv, P, d = codes.shape
    x = x.float()
    page, slot = page.long(), slot.long()
    first = torch.full((num_pages,), P, dtype=torch.int64, device="cuda").scatter_reduce(0, page, slot, "amin")
    amax = torch.zeros((num_pages, Hkv), device="cuda").scatter_reduce(0, page[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
    old = torch.where(first[:, None] > 0, scales, 0.0)
    touched = first < P
    scale = torch.where(touched[:, None], torch.maximum(old, _pow2_scale(amax)), scales)
    inverse = torch.where(scale > 0, 1.0 / scale, 0.0)
    older = torch.nonzero(touched & (first > 0))[:, 0]
    had = codes[older]
    again = _encode(_values(had) * (old * inverse)[older][:, :, None, None])
    keep = torch.arange(P, device="cuda")[None, None, :, None] < first[older][:, None, None, None]
    codes[older] = torch.where(keep, again, had)
    codes[page, :, slot] = _encode(x * inverse[page][:, :, None])
    scales.copy_(scale)


def _run_append(s, c):
    if own:
        _ops().kv8_append(s["k_new"], s["v_new"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["page"], s["slot"])
    else:
        _append_one(s["k_new"], s["k_codes"], s["k_scale"], s["page"], s["slot"])
        _append_one(s["v_new"], s["v_codes"], s["v_scale"], s["page"], s["slot"])
    return s["k_codes"].view(torch.float8_e4m3fn), s["v_codes"].view(torch.float8_e4m3fn), s["k_scale"], s["v_scale"]


def _run_decode(s, c):
    if own:
        return _ops().decode_kv8(s["q"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["table"], s["seq_lens"],
                                 c["L_hi"], window_left=c["window"])
    B, Nq, Hq, d = s["q"].shape
    Hkv, P = c["Hkv"], c["P"]
    group, L = Hq // Hkv, s["table"].shape[1] * P
    table, lens = s["table"].long(), s["seq_lens"].long()
    j = torch.arange(L, device="cuda")[None]

    def keys(codes, scales):  # [B, Hkv, L, d]; what lies behind a request's last key counts as zero
        x = (_values(codes[table]) * scales[table][..., None, None]).transpose(1, 2).reshape(B, Hkv, L, d)
        return x.masked_fill_((j >= lens[:, None])[:, None, :, None], 0.0)

    q = s["q"].float().reshape(B, Nq, Hkv, group, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, group * Nq, d)
    score = (q @ keys(s["k_codes"], s["k_scale"]).transpose(2, 3)).view(B, Hkv, group, Nq, L) * d ** -0.5
    at = lens[:, None] - Nq + torch.arange(Nq, device="cuda")[None]
    seen = (j[:, None] <= at[..., None]) & (j[:, None] < lens[:, None, None])
    if c["window"] >= 0:
        seen &= j[:, None] >= at[..., None] - c["window"]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = (score - top).exp()
    total = weight.sum(-1, keepdim=True)
    o = (weight.view(B, Hkv, group * Nq, L) @ keys(s["v_codes"], s["v_scale"])).view(B, Hkv, group, Nq, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + total.log())[..., 0].reshape(B, Hq, Nq)
    return o.permute(0, 3, 1, 2, 4).reshape(B, Nq, Hq, d).to(torch.bfloat16), lse


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "plan":
        new = _spread(c["new_lo"], c["new_hi"], c["B"])
        rows = sum(new) + c["pad"]
        return {"bytes": 4 * (2 * c["B"] + 2 * (sum(new) // c["P"] + 1) + 2 * c["B"] + 1 + 3 * rows), "flops": 0}
    if c["op"] == "rope":
        n = c["T"] * (c["Hq"] + c["Hkv"]) * c["d"]
        return {"bytes": 4 * n + 4 * c["n_axes"] * c["T"], "flops": 3 * n}
    if c["op"] == "append":
        n = c["B"] * c["new"]
        return {"bytes": 2 * n * c["Hkv"] * c["d"] * 3 + 8 * n + 16 * c["Hkv"] * (n // c["P"] + c["B"]), "flops": 4 * n * c["Hkv"] * c["d"]}
    lens = _spread(c["L_lo"], c["L_hi"], c["B"])
    seen = [min(n, c["window"] + c["Nq"]) if c["window"] >= 0 else n for n in lens]
    keys, rows = sum(seen) * c["Hkv"], c["B"] * c["Nq"] * c["Hq"]
    pairs = sum(sum(max(0, min(n - c["Nq"] + i + 1, c["window"] + 1 if c["window"] >= 0 else n)) for i in range(c["Nq"])) for n in lens)
    return {"bytes": 2 * keys * c["d"] + 8 * keys // c["P"] + 4 * sum(seen) // c["P"] + rows * (4 * c["d"] + 4),
            "flops": 4 * pairs * c["Hq"] * c["d"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": lambda s: None, "rope": _exact_rope, "append": _exact_append, "decode": _exact_decode}[case["op"]](s)


def _exact_rope(s):
    """Each pair as a complex number times e^(i angle)."""
    c, half = s["case"], s["case"]["d"] // 2
    angle = torch.stack([s["positions"][int(a)].double() for a in s["axis"].tolist()], dim=1) * s["freq"]
    turn = torch.polar(torch.ones_like(angle), -angle if c["bwd"] else angle)[:, None]
    out = []
    for x in (s["q"].double(), s["k"].double()):
        pairs = x.unflatten(-1, (half, 2)) if c["neighbours"] else x.unflatten(-1, (2, half)).transpose(-1, -2)
        r = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        out.append((r if c["neighbours"] else r.transpose(-1, -2)).flatten(-2))
    return tuple(out)


def _exact_append(s):
    """Page by page: what each code would be without its last rounding."""
    if s["page"].numel() // s["case"]["P"] + s["case"]["B"] > 20000:
        return None
    got = []
    page, slot = s["page"].long(), s["slot"].long()
    for x, codes, scales in ((s["k_new"], s["k_codes"], s["k_scale"]), (s["v_new"], s["v_codes"], s["v_scale"])):
        want, size = _values(codes).double(), scales.double()
        order = torch.argsort(page, stable=True)
        pages, counts = torch.unique_consecutive(page[order], return_counts=True)
        at = 0
        for p, n in zip(pages.tolist(), counts.tolist()):
            rows = order[at: at + n]
            at += n
            first = slot[rows].min()
            x64 = x[rows].double()
            loudest = x64.abs().amax(dim=(0, 2))
            need = torch.where(loudest > 0, torch.exp2(torch.ceil(torch.log2(loudest / 448.0))), 0.0)
            old = torch.where(first > 0, size[p], torch.zeros_like(size[p]))
            new = torch.maximum(old, need)
            before = (torch.arange(codes.shape[2], device="cuda") < first)[None, :, None]
            want[p] = torch.where(before, want[p] * (old / new)[:, None, None], want[p])
            want[p][:, slot[rows]] = (x64 / new[None, :, None]).transpose(0, 1)
            size[p] = new
        got.append((want, size))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def _exact_decode(s):
    """Request by request, the cache read back as numbers."""
    c = s["case"]
    B, Nq, Hq, d = s["q"].shape
    Hkv, P = c["Hkv"], c["P"]
    o = torch.zeros((B, Nq, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["seq_lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, : -(-n // P)].long()
        k, v = ((_values(x[pages]).double() * y[pages].double()[..., None, None]).transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
                for x, y in ((s["k_codes"], s["k_scale"]), (s["v_codes"], s["v_scale"])))
        for i in range(Nq):
            hi = n - Nq + i + 1
            lo = max(0, hi - 1 - c["window"]) if c["window"] >= 0 else 0
            if hi <= lo:
                continue
            q = s["q"][b, i].double().view(Hkv, Hq // Hkv, d)
            score = torch.einsum("hgd,hjd->hgj", q, k[:, lo:hi]) / math.sqrt(d)
            lse[b, :, i] = torch.logsumexp(score, -1).flatten()
            o[b, i] = torch.einsum("hgj,hjd->hgd", torch.softmax(score, -1), v[:, lo:hi]).reshape(Hq, d)
    return o, lse
