"""The measured cases of the sampling-step operators: norms of query and key
heads with the position rotation in the same pass and their gradients, and the
attention of a batch whose requests share long prefixes, over the bf16 pages
and over the 8-bit ones; each with its plain form in elementary torch
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
        # norm and rotation of one decode step: latency
        dict(name="norm decode step", op="norm", T=64, Hq=32, Hkv=8, d=128, n_axes=1, neighbours=0, wide=0, bwd=0),
        # a long prompt or a training batch
        dict(name="norm prompt", op="norm", T=16384, Hq=32, Hkv=8, d=128, n_axes=1, neighbours=0, wide=0, bwd=0),
        # the same batch's gradients, odd length
        dict(name="norm gradient", op="norm", T=16383, Hq=32, Hkv=8, d=128, n_axes=1, neighbours=0, wide=1, bwd=1),
        # training on video patches: three axes, neighbouring pairs, narrow heads
        dict(name="norm video gradient", op="norm", T=12289, Hq=16, Hkv=16, d=64, n_axes=3, neighbours=1, wide=0, bwd=1),
        # four answers to one short question: latency
        dict(name="shared four answers", op="shared", kv8=0, G=1, n=4, Nq=1, Hq=32, Hkv=8, d=128, Ls_lo=777, Ls_hi=777,
             own_lo=1, own_hi=64, P=16, window=-1),
        # a server whose requests share a long system prompt
        dict(name="shared system prompt", op="shared", kv8=0, G=1, n=64, Nq=1, Hq=64, Hkv=8, d=128, Ls_lo=16385, Ls_hi=16385,
             own_lo=100, own_hi=2000, P=16, window=-1),
        # many samples of one long document, as search over answers and policy training draw them
        dict(name="shared many samples", op="shared", kv8=0, G=1, n=256, Nq=1, Hq=64, Hkv=8, d=128, Ls_lo=32768, Ls_hi=32768,
             own_lo=1, own_hi=512, P=64, window=-1),
        # several prompts, eight samples each, one K/V head for each query head
        dict(name="shared sampled prompts", op="shared", kv8=0, G=16, n=8, Nq=1, Hq=16, Hkv=16, d=64, Ls_lo=500, Ls_hi=8000,
             own_lo=1, own_hi=1000, P=32, window=-1),
        # drafts verified over a shared prompt, a sliding-window layer
        dict(name="shared drafts window", op="shared", kv8=0, G=2, n=16, Nq=4, Hq=32, Hkv=8, d=128, Ls_lo=4001, Ls_hi=9001,
             own_lo=4, own_hi=300, P=16, window=4095),
        # the 8-bit cache: the short question, the system prompt, the long document
        dict(name="shared8 four answers", op="shared", kv8=1, G=1, n=4, Nq=1, Hq=32, Hkv=8, d=128, Ls_lo=777, Ls_hi=777,
             own_lo=1, own_hi=64, P=16, window=-1),
        dict(name="shared8 system prompt", op="shared", kv8=1, G=1, n=64, Nq=1, Hq=64, Hkv=8, d=128, Ls_lo=16385, Ls_hi=16385,
             own_lo=100, own_hi=2000, P=16, window=-1),
        dict(name="shared8 many samples", op="shared", kv8=1, G=1, n=256, Nq=1, Hq=64, Hkv=8, d=128, Ls_lo=32768, Ls_hi=32768,
             own_lo=1, own_hi=512, P=64, window=-1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["norm", "shared", "shared"])
    if op == "norm":
        Hkv = rng.choice([1, 2, 4, 8, 16])
        Hq = Hkv * rng.choice([1, 2, 4, 7])
        d = rng.choice([64, 128])
        T = _log(rng, 1, max(1, min(65536, 80000000 // (d * (Hq + Hkv)))))
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, d=d, n_axes=rng.choice([1, 2, 3]), neighbours=rng.choice([0, 1]),
                    wide=rng.choice([0, 1]), bwd=rng.choice([0, 1]))
    Hkv, d = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128])
    Nq, Hq = rng.choice([1, 1, 1, 2, 4]), Hkv * rng.choice([1, 2, 4, 5, 8])
    G = _log(rng, 1, 16)
    n = _log(rng, 1, 256 // G)
    Ls = _log(rng, 1, max(1, min(65536, 400000000 // (G * Hkv * d), 60000000000 // (G * n * Nq * Hq * d))))
    hi = _log(rng, Nq, max(Nq, min(4096, 200000000 // (G * n * Hkv * d), 10000000000 // (G * n * Nq * Hq * d))))
    return dict(op=op, kv8=rng.choice([0, 1]), G=G, n=n, Nq=Nq, Hq=Hq, Hkv=Hkv, d=d, Ls_lo=rng.choice([Ls, Ls, max(1, Ls // 5)]),
                Ls_hi=Ls, own_lo=rng.choice([Nq, hi]), own_hi=hi, P=rng.choice([16, 32, 64, 128]),
                window=rng.choice([-1, -1, -1, Ls // 2, 1023]))


def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spread: their sum does not depend on the seed, their order does."""
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _shared_lens(c):
    """Tokens that each group shares; of the 8-bit cache whole pages, whose scales are then one."""
    return [n // c["P"] * c["P"] if c["kv8"] else n for n in _spread(c["Ls_lo"], c["Ls_hi"], c["G"])]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _loud(d, g):
    """Keys have a few loud channels, as trained models' keys do."""
    loud = torch.ones(d, device="cuda")
    loud[torch.randperm(d, generator=g, device="cuda")[: d // 16]] = 3.0
    return loud


def _pages(num_pages, P, Hkv, d, g, loud):
    """[num_pages, P, Hkv, d] bf16."""
    pages = torch.empty((num_pages, P, Hkv, d), dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 27) // (Hkv * P * d))
    for a in range(0, num_pages, step):
        pages[a:a + step] = torch.randn(pages[a:a + step].shape, generator=g, device="cuda") * loud
    return pages


def _pages8(num_pages, P, Hkv, d, g, loud):
    """e4m3 codes [num_pages, Hkv, P, d] and a power of two for each page and head."""
    codes = torch.empty((num_pages, Hkv, P, d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((num_pages, Hkv), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (Hkv * P * d))
    for a in range(0, num_pages, step):
        x = torch.randn(codes[a:a + step].shape, generator=g, device="cuda") * loud
        m, e = torch.frexp(x.abs().amax(dim=(2, 3)) / 448.0)
        s = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))
        codes[a:a + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[a:a + step] = s
    return codes, scales


def prepare(case, seed):
    return (_prepare_norm if case["op"] == "norm" else _prepare_shared)(dict(case), _gen(seed))


def _frequencies(c):
    """(axis of each pair, frequency of each pair) as plain lists."""
    half, A = c["d"] // 2, c["n_axes"]
    sizes = [half] if A == 1 else [half // 2, half - half // 2] if A == 2 else [half // 4, half // 8 * 3, half - half // 4 - half // 8 * 3]
    return [a for a in range(A) for _ in range(sizes[a])], [1000000.0 ** (-i / half) for i in range(half)]


def _prepare_norm(c, g):
    T, Hq, Hkv, d, A = c["T"], c["Hq"], c["Hkv"], c["d"], c["n_axes"]
    # q, k and v come out of one projection: rows of q and k are slices of its rows; heads differ in size
    size = torch.exp(torch.randn((Hq + 2 * Hkv, 1), generator=g, device="cuda") * 0.7)
    qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=g, device="cuda").mul_(size).to(torch.bfloat16)
    t = torch.arange(T, device="cuda")
    start = torch.randint(0, 100000, (1,), generator=g, device="cuda")
    text = T // 4  # text first, then patches of 24 x 32 frames
    patch = (t - text).clamp(min=0)
    grid = torch.stack([patch // 768, patch // 32 % 24, patch % 32])[-A:] + text if A > 1 else t[None]
    pos = torch.where(t < text, t[None].expand(A, T), grid) + start
    axis, freq = _frequencies(c)
    s = dict(case=c, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], positions=pos.to(torch.int32).contiguous(), eps=1e-6,
             axis=torch.tensor(axis, device="cuda"), freq=torch.tensor(freq, dtype=torch.float64, device="cuda"))
    for name in ("wq", "wk"):  # trained weights of a norm lie around one
        w = 1 + 0.25 * torch.randn(d, generator=g, device="cuda")
        s[name] = w if c["wide"] else w.to(torch.bfloat16)
    if c["bwd"]:
        s["dq"] = torch.randn((T, Hq, d), generator=g, device="cuda").to(torch.bfloat16)
        s["dk"] = torch.randn((T, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    if own:
        s["plan"] = _ops().RopePlan(d, axis, freq, neighbours=bool(c["neighbours"]))
    return s


def _prepare_shared(c, g):
    G, n, P, Hkv, d = c["G"], c["n"], c["P"], c["Hkv"], c["d"]
    B = G * n
    shared = torch.tensor(_shared_lens(c), device="cuda")
    lens = torch.tensor(_spread(c["own_lo"], c["own_hi"], B), device="cuda")
    lens = lens[torch.randperm(B, generator=g, device="cuda")] + shared.repeat_interleave(n)
    full = shared // P  # pages that a group's tables have in common; a partly filled one each request has for itself
    first = torch.cumsum(full, 0) - full
    blocks = (lens + P - 1) // P
    mine = blocks - full.repeat_interleave(n)
    start = torch.cumsum(mine, 0) - mine + full.sum()
    num_pages = sum(x // P for x in _shared_lens(c)) + sum(x // P + 2 for x in _spread(c["own_lo"], c["own_hi"], B)) + 3
    order = torch.randperm(num_pages, generator=g, device="cuda")
    max_len = max(_shared_lens(c)) + c["own_hi"]
    cols = torch.arange(-(-max_len // P), device="cuda")[None]
    own_col = cols - full.repeat_interleave(n)[:, None]
    at = torch.where(own_col < 0, first.repeat_interleave(n)[:, None] + cols, start[:, None] + own_col)
    table = torch.where(cols < blocks[:, None], order[at.clamp(max=num_pages - 1)], 0)
    s = dict(case=c, seq_lens=lens.to(torch.int32), table=table.to(torch.int32).contiguous(), max_len=max_len,
             shared_lens=shared.to(torch.int32), group_starts=torch.arange(0, B + 1, n, dtype=torch.int32, device="cuda"))
    loud = _loud(d, g)
    if c["kv8"]:
        s["k"], s["k_scale"] = _pages8(num_pages, P, Hkv, d, g, loud)
        s["v"], s["v_scale"] = _pages8(num_pages, P, Hkv, d, g, 1.0)
    else:
        s["k"], s["v"] = _pages(num_pages, P, Hkv, d, g, loud), _pages(num_pages, P, Hkv, d, g, 1.0)
        for i, x in enumerate(_shared_lens(c)):  # the partly filled page was copied for each request
            if x % P:
                pages = table[i * n:(i + 1) * n, x // P]
                for t in (s["k"], s["v"]):
                    t[pages, :x % P] = t[pages[0], :x % P]
    s["q"] = (1.5 * torch.randn((B, c["Nq"], c["Hq"], d), generator=g, device="cuda")).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_run_norm if s["case"]["op"] == "norm" else _run_shared)(s, s["case"])


def _rotate(x, ca, sa, neighbours):
    """x [T, H, d] in 32 or 64 bits; ca, sa [T, 1, d / 2]."""
    if neighbours:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * ca - b * sa, a * sa + b * ca], dim=-1).flatten(-2)
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * ca - b * sa, a * sa + b * ca], dim=-1)


def _run_norm(s, c):
    if own:
        if c["bwd"]:
            return _ops().qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["plan"],
                                           eps=s["eps"])
        return _ops().qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["plan"], eps=s["eps"])
    angle = s["positions"].t()[:, s["axis"]].double() * s["freq"]
    ca, sa = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out, grads = [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x, w = x.float(), w.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
        n = x * r
        if not c["bwd"]:
            out.append(_rotate(n * w, ca, sa, c["neighbours"]).to(torch.bfloat16))
            continue
        dy = _rotate(dy.float(), ca, -sa, c["neighbours"])
        grads.append((dy * n).sum((0, 1)))
        dn = dy * w
        out.append((r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(torch.bfloat16))
    return tuple(out + grads)


def _run_shared(s, c):
    if own:
        tail = (s["table"], s["seq_lens"], s["group_starts"], s["shared_lens"], s["max_len"])
        if c["kv8"]:
            return _ops().decode_kv8_shared(s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], *tail, window_left=c["window"])
        return _ops().decode_paged_shared(s["q"], s["k"], s["v"], *tail, window_left=c["window"])
    n, P, Nq, Hq, Hkv, d = (c[x] for x in ("n", "P", "Nq", "Hq", "Hkv", "d"))
    rows, L = Hq // Hkv * Nq, c["own_hi"]
    out, sums = [], []

    def cached(side, pages):  # [pages ..., Hkv, P, d]
        if c["kv8"]:
            return _values(s[side][pages]) * s[side + "_scale"][pages][..., None, None]
        return s[side][pages].float().transpose(-3, -2)

    for i, m in enumerate(_shared_lens(c)):  # a group's shared keys meet the queries of all its requests at once
        table, lens = s["table"][i * n:(i + 1) * n].long(), s["seq_lens"][i * n:(i + 1) * n].long()
        pages = table[0, : -(-m // P)]
        j = m + torch.arange(L, device="cuda")[None]  # positions of each request's own keys
        blk = (m // P + torch.arange(L // P + 2, device="cuda")).clamp(max=table.shape[1] - 1)
        at = m % P + torch.arange(L, device="cuda")
        gone = (j >= lens[:, None])[:, None, :, None]

        def keys(side):
            a = cached(side, pages).transpose(0, 1).reshape(Hkv, -1, d)[:, :m]
            b = cached(side, table[:, blk]).transpose(1, 2).reshape(n, Hkv, -1, d)[:, :, at].masked_fill(gone, 0.0)
            return a, b

        q = s["q"][i * n:(i + 1) * n].float().view(n, Nq, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(n, Hkv, rows, d)
        k, k_own = keys("k")
        score = torch.cat([(q.transpose(0, 1).reshape(Hkv, n * rows, d) @ k.transpose(1, 2)).view(Hkv, n, rows, m).transpose(0, 1),
                           q @ k_own.transpose(2, 3)], dim=-1).mul_(d ** -0.5)
        pos = torch.arange(m + L, device="cuda")
        stand = lens[:, None] - Nq + torch.arange(Nq, device="cuda")[None]
        seen = pos <= stand[..., None]  # [n, Nq, keys]
        if c["window"] >= 0:
            seen &= pos >= stand[..., None] - c["window"]
        score.view(n, Hkv, Hq // Hkv, Nq, m + L).masked_fill_(~seen[:, None, None], -math.inf)
        top = score.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        weight = score.sub_(top).exp_()
        total = weight.sum(-1, keepdim=True)
        v, v_own = keys("v")
        o = (weight[..., :m].transpose(0, 1).reshape(Hkv, n * rows, m) @ v).view(Hkv, n, rows, d).transpose(0, 1) + weight[..., m:] @ v_own
        o = torch.where(total > 0, o / total, 0.0)
        out.append(o.view(n, Hq, Nq, d).transpose(1, 2).to(torch.bfloat16))
        sums.append((top + total.log())[..., 0].reshape(n, Hq, Nq))
    return torch.cat(out), torch.cat(sums)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * (c["Hq"] + c["Hkv"]) * c["d"]
        return {"bytes": (6 if c["bwd"] else 4) * n + 4 * c["n_axes"] * c["T"] + (12 if c["bwd"] else 4) * c["d"],
                "flops": (16 if c["bwd"] else 8) * n}
    n, Nq, w = c["n"], c["Nq"], c["window"]
    B = c["G"] * n
    own_lens = _spread(c["own_lo"], c["own_hi"], B)
    keys = pairs = 0
    for i, m in enumerate(_shared_lens(c)):
        # (which request has which length is the seed's; a window's share is counted with the group's mean)
        mean = sum(own_lens) // B
        keys += min(m, max(0, w + Nq - min(own_lens))) if w >= 0 else m
        for a in own_lens[i * n:(i + 1) * n]:
            keys += min(a, w + Nq) if w >= 0 else a
            for x in range(Nq):
                at = m + (mean if w >= 0 else a) - Nq + x + 1
                pairs += min(at, w + 1) if w >= 0 else at
    size = (2 * c["d"] + 8 / c["P"]) if c["kv8"] else 4 * c["d"]
    rows = B * Nq * c["Hq"]
    return {"bytes": int(keys * c["Hkv"] * size) + rows * (4 * c["d"] + 4) + 4 * keys // c["P"], "flops": 4 * pairs * c["Hq"] * c["d"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_norm if case["op"] == "norm" else _exact_shared)(s, case)


def _exact_norm(s, c):
    """Heads divided by their root mean square; each pair as a complex number times e^(i angle).  Token blocks."""
    half, nb = c["d"] // 2, c["neighbours"]
    outs = [[], []]
    sums = [torch.zeros(c["d"], dtype=torch.float64, device="cuda") for _ in range(2)]

    def turned(x, turn):
        pairs = x.unflatten(-1, (half, 2)) if nb else x.unflatten(-1, (2, half)).transpose(-1, -2)
        r = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        return (r if nb else r.transpose(-1, -2)).flatten(-2)

    for t in range(0, c["T"], 4096):
        rows = slice(t, t + 4096)
        angle = s["positions"][:, rows].double()[s["axis"]].t() * s["freq"]
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        for i, (x, w, dy) in enumerate(((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk")))):
            x, w = x[rows].double(), w.double()
            rms = (x.pow(2).sum(-1, keepdim=True) / c["d"] + s["eps"]).sqrt()
            if not c["bwd"]:
                outs[i].append(turned(x / rms * w, turn))
                continue
            dy = turned(dy[rows].double(), turn.conj())
            sums[i] += (dy * x / rms).sum((0, 1))
            dn = dy * w
            outs[i].append(dn / rms - x * (dn * x).sum(-1, keepdim=True) / (c["d"] * rms.pow(3)))
    outs = [torch.cat(x) for x in outs]
    return tuple(outs + sums) if c["bwd"] else tuple(outs)


def _exact_shared(s, c):
    """Request by request over its whole row of the table, the cache read back as numbers."""
    n, P, Nq, Hq, Hkv, d = (c[x] for x in ("n", "P", "Nq", "Hq", "Hkv", "d"))
    if c["G"] * n * Nq * Hq * c["Ls_hi"] * d > 2e12:
        return None
    o = torch.zeros((c["G"] * n, Nq, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((c["G"] * n, Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["seq_lens"].tolist()):
        least = max(0, length - Nq - c["window"]) // P if c["window"] >= 0 else 0  # the first page any query sees
        pages = s["table"][b, least: -(-length // P)].long()
        if c["kv8"]:
            k, v = ((_values(s[x][pages]).double() * s[x + "_scale"][pages].double()[..., None, None]).transpose(0, 1)
                    .reshape(Hkv, -1, d) for x in ("k", "v"))
        else:
            k, v = (s[x][pages].double().flatten(0, 1).transpose(0, 1) for x in ("k", "v"))
        for i in range(Nq):
            hi = length - Nq + i + 1
            lo = max(0, hi - 1 - c["window"]) if c["window"] >= 0 else 0
            if hi <= lo:
                continue
            part = slice(lo - least * P, hi - least * P)
            score = torch.einsum("hgd,hjd->hgj", s["q"][b, i].double().view(Hkv, Hq // Hkv, d), k[:, part]) / math.sqrt(d)
            lse[b, :, i] = torch.logsumexp(score, -1).flatten()
            o[b, i] = torch.einsum("hgj,hjd->hgd", torch.softmax(score, -1), v[:, part]).reshape(Hq, d)
    return o, lse
