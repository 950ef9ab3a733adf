"""Filtered sampling and the bounded drafter cache, as cases to measure.

Four operators in two pairs, next to the greedy readout, the rejection
sampling and the 4-bit paged cache:

  sample   draft tokens from logits rows under temperature, top-k, top-p and
           min-p, one given uniform number a row
  verify   rejection sampling of drafts against the same filtered
           distributions, from given coins and one given number a request
  weigh    attention weight that every cached key gets from a step's rows,
           added to what it had
  evict    the heaviest keys of each request and key head, gathered at the
           front of the destination pages

A row's filter: y = x / T; columns by y descending, equal ones by column; the
first k of them; of those the smallest prefix whose weight is at least top_p of
theirs; of those the ones of at least min_p of the largest weight.  T = 0
keeps the first column alone.  The token is the first column, in column
order, whose running sum of kept weights exceeds u times their sum.

The cache is one byte tensor [num_blocks, Hkv, block_size / 16, 18 D]: a record
holds 16 tokens' key codes [16][D/2], value codes [16][D/2], key scales
[16][D/16] and value scales [16][D/16]; a code is an e2m1 number (element 2i
in the low half of byte i), a scale an e4m3 number shared by 16 elements.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# (temperature, top_k, top_p, min_p) as requests ask for them; k = 0, p = 1 and 0 are "off"
ASKED = {
    "chat": [(0.7, 20, 0.8, 0.0)],
    "nucleus": [(0.8, 0, 0.95, 0.0)],
    "open": [(1.0, 0, 1.0, 0.0)],
    "minp": [(1.3, 0, 1.0, 0.05)],
    "mixed": [(0.7, 20, 0.8, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.6, 64, 0.95, 0.0), (0.9, 0, 0.9, 0.02),
              (1.0, 1, 1.0, 0.0), (1.2, 0, 1.0, 0.1), (0.8, 200, 0.99, 0.0)],
}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the drafter of one stream: seven rows, latency counts
        dict(name="sample b1", op="sample", B=1, K=7, V=201088, fp32=False, asked="chat"),
        # fp32 logits without any filter: every column counts
        dict(name="sample open fp32 b16", op="sample", B=16, K=3, V=201088, fp32=True, asked="open"),
        # the large serving batch, requests that ask for different things
        dict(name="sample b256", op="sample", B=256, K=7, V=151936, fp32=False, asked="mixed"),
        # one stream's verification: 8 target rows, 7 draft rows
        dict(name="verify b1", op="verify", B=1, Kp=7, V=201088, fp32=False, asked="chat"),
        # the middle serving batch, nucleus sampling
        dict(name="verify b64", op="verify", B=64, Kp=7, V=201088, fp32=False, asked="nucleus"),
        # the large serving batch
        dict(name="verify b256", op="verify", B=256, Kp=7, V=151936, fp32=False, asked="mixed"),
        # one stream, one token: the smallest call over a cache
        dict(name="weigh token b1", op="weigh", B=1, Kp=0, K=1, lo=4000, hi=4000, Hq=64, Hkv=8, D=64, bs=16),
        # the middle serving batch's draft rows
        dict(name="weigh draft b64", op="weigh", B=64, Kp=7, K=7, lo=256, hi=32767, Hq=64, Hkv=8, D=64, bs=16),
        # the large serving batch, one token a request
        dict(name="weigh token b256", op="weigh", B=256, Kp=0, K=1, lo=0, hi=65535, Hq=32, Hkv=4, D=128, bs=16),
        # one stream over its budget by a page's worth of keys
        dict(name="evict b1", op="evict", B=1, lo=1040, hi=1040, keep=1024, sinks=4, recent=64, Hkv=8, D=64, bs=16),
        # long prompts cut to a budget right after prefill
        dict(name="evict b8", op="evict", B=8, lo=20000, hi=65535, keep=4096, sinks=4, recent=512, Hkv=8, D=64, bs=16),
        # the large serving batch; requests below the budget stay whole
        dict(name="evict b256", op="evict", B=256, lo=0, hi=32767, keep=2048, sinks=4, recent=256, Hkv=4, D=128, bs=16),
    ]


HEADS = ((64, 8, 64), (32, 4, 128), (32, 8, 128), (12, 12, 64), (20, 4, 64), (8, 1, 128))


def draw(rng):
    def span(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("sample", "verify", "weigh", "evict"))
    if op in ("sample", "verify"):
        V = span(100, 201088)
        c = dict(op=op, B=span(1, min(256, 12_000_000 // V)), V=V, fp32=rng.random() < 0.3, asked=rng.choice(sorted(ASKED)))
        c["K" if op == "sample" else "Kp"] = rng.randint(1, 7)
        return c
    Hq, Hkv, D = rng.choice(HEADS)
    bs = rng.choice((16, 16, 32, 64))
    B = span(1, 256)
    hi = span(16, min(65535, 2_000_000 // B))
    c = dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, Hkv=Hkv, D=D, bs=bs)
    if op == "weigh":
        draft = rng.random() < 0.5
        c.update(Hq=Hq, Kp=rng.randint(1, 7) if draft else 0, K=rng.randint(1, 7) if draft else 1)
    else:
        keep = span(1, min(8192, 2 * hi))
        c.update(keep=keep, sinks=rng.randint(0, min(8, keep)), recent=rng.randint(0, keep // 2))
    return c


def _spread(i, lo, hi):
    """The i-th of evenly spread whole numbers of [lo, hi] (a fixed sequence: work() needs it too)."""
    return lo + int((hi - lo + 1) * math.fmod((i + 1) * 0.6180339887498949, 1.0))


def _rows(c):
    """(position, kept) of the packed rows of each request, as the draft-batch rebuild lays them out: the verified
    rows (those after the bonus slot are rejected), then K-1 MASK rows from the bonus slot's position on."""
    rows = []
    for b in range(c["B"]):
        first = _spread(b, c["lo"], c["hi"])
        a = min(c["Kp"], int(-math.log(1.0 - math.fmod((b + 1) * 0.7548776662466927, 1.0)) * 2))
        rows.append([(first + k, k <= a) for k in range(c["Kp"] + 1)] + [(first + a + i, True) for i in range(1, c["K"])])
    return rows


def _lengths(c):
    return [_spread(b, c["lo"], c["hi"]) for b in range(c["B"])]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"sample": _prepare_sample, "verify": _prepare_verify, "weigh": _prepare_weigh, "evict": _prepare_evict}[case["op"]](case, g)


def _logits(case, n, g, like=None):
    """Rows of a language model's logits: a wide bulk, and a few hundred plausible tokens that fall off as a power of
    their rank; rows are padded to whole 16-byte vectors, as an LM head's output is.  ``like``: rows of a model
    that tells nearly the same."""
    V = case["V"]
    pitch = -(-V // 8) * 8
    out = torch.full((n, pitch), 3.0e38, dtype=torch.float32 if case["fp32"] else torch.bfloat16, device="cuda")
    if like is not None:
        out[:, :V] = like.float() + 0.5 * torch.randn(n, V, generator=g, device="cuda")
        return out[:, :V]
    x = 2.0 * torch.randn(n, V, generator=g, device="cuda")
    m = min(300, V)
    rank = torch.arange(1, m + 1, device="cuda", dtype=torch.float32)
    steep = 1.0 + torch.rand(n, 1, generator=g, device="cuda")
    top = 16.0 + 2.0 * torch.rand(n, 1, generator=g, device="cuda") - steep * rank.log()
    at = torch.randint(0, V, (n, m), generator=g, device="cuda")
    x.scatter_reduce_(1, at, top + 0.5 * torch.randn(n, m, generator=g, device="cuda"), "amax")  # (columns may repeat)
    out[:, :V] = x
    return out[:, :V]


def _asked(case):
    """Per-request parameters."""
    rows = ASKED[case["asked"]]
    t, k, p, m = zip(*[rows[b % len(rows)] for b in range(case["B"])])
    f = lambda v, dt=torch.float32: torch.tensor(v, dtype=dt, device="cuda")  # noqa: E731
    return dict(temperature=f(t), top_k=f(k, torch.int32), top_p=f(p), min_p=f(m))


def _prepare_sample(case, g):
    n = case["B"] * case["K"]
    s = dict(case=case, logits=_logits(case, n, g), asked=_asked(case), u=torch.rand(n, generator=g, device="cuda"),
             tokens=torch.empty(n, dtype=torch.int32, device="cuda"), prob=torch.empty(n, device="cuda"))
    return _plan(s)


def _prepare_verify(case, g):
    B, Kp = case["B"], case["Kp"]
    target = _logits(case, B * (Kp + 1), g)
    drafted = (torch.arange(B * (Kp + 1), device="cuda") % (Kp + 1)) < Kp
    draft = _logits(case, B * Kp, g, like=target[drafted])
    asked = _asked(case)
    w = _kept_weights(draft, {n: v.repeat_interleave(Kp) for n, v in asked.items()})
    tokens = torch.zeros(B, Kp + 1, dtype=torch.int32, device="cuda")
    tokens[:, 1:] = _drawn(w, torch.rand(B * Kp, generator=g, device="cuda")).view(B, Kp)
    s = dict(case=case, target=target, draft=draft, asked=asked, tokens=tokens.flatten(),
             coins=torch.rand(B * Kp, generator=g, device="cuda"), u=torch.rand(B, generator=g, device="cuda"),
             accepted=torch.empty(B, dtype=torch.int32, device="cuda"), bonus=torch.empty(B, dtype=torch.int32, device="cuda"),
             chance=torch.empty(B * Kp, device="cuda"))
    return _plan(s)


def _pages(case, need, width, g, spare=0):
    """A block table whose pages lie in a random order, and spare pages after them."""
    perm = torch.randperm(sum(need) + spare, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(need), width, dtype=torch.int32, device="cuda")
    at = torch.tensor([0] + need, device="cuda").cumsum(0)
    col = torch.arange(width, device="cuda")
    live = col < at.diff()[:, None]
    table[live] = perm[(at[:-1, None] + col)[live]]
    return table, perm[sum(need):]


def _random_cache(case, blocks, g):
    """Codes of values of a projection's size, with the scales that 16 normal numbers have."""
    Hkv, D, bs = case["Hkv"], case["D"], case["bs"]
    cache = torch.empty(blocks, Hkv, bs // 16, 18 * D, dtype=torch.uint8, device="cuda")
    cache[..., :16 * D] = torch.randint(0, 256, (blocks, Hkv, bs // 16, 16 * D), generator=g, device="cuda", dtype=torch.uint8)
    for at in (16 * D, 17 * D):
        s = 0.2 + 0.4 * torch.rand(blocks, Hkv, bs // 16, D, generator=g, device="cuda")
        cache[..., at:at + D] = s.to(torch.float8_e4m3fn).view(torch.uint8)
    return cache


def _prepare_weigh(case, g):
    Hq, Hkv, D, bs, rows = case["Hq"], case["Hkv"], case["D"], case["bs"], _rows(case)
    most = [max(p for p, k in r if k) + 1 for r in rows]
    need = [-(-n // bs) for n in most]
    s = dict(case=case, scale=1.0 / math.sqrt(D), longest=max(most), m=len(rows[0]))
    s["block_table"], _ = _pages(case, need, max(need) + 1, g)
    s["cache"] = _random_cache(case, sum(need), g)
    s["positions"] = torch.tensor([p for r in rows for p, _ in r], dtype=torch.int32, device="cuda")
    s["is_rejected"] = torch.tensor([not k for r in rows for _, k in r], dtype=torch.uint8, device="cuda")
    T = len(rows) * s["m"]
    q = torch.randn(T, Hq * D, generator=g, device="cuda")
    q *= 1.0 + 2.0 * (torch.rand(Hq * D, generator=g, device="cuda") > 0.97)
    s["q"] = q.to(torch.bfloat16).view(T, Hq, D)
    # what some sixteen earlier steps left; the rows' own keys are new and start from nothing
    s["mass"] = torch.rand(sum(need), Hkv, bs, generator=g, device="cuda").pow(8) * (144.0 * Hq / Hkv / max(most))
    s["fresh"] = torch.tensor([min(p for p, _ in r) for r in rows], dtype=torch.int32, device="cuda")
    s["out"] = torch.zeros_like(s["mass"])
    return _plan(s)


def _prepare_evict(case, g):
    B, Hkv, bs = case["B"], case["Hkv"], case["bs"]
    lens = _lengths(case)
    width = -(-case["keep"] // bs)
    s = dict(case=case, longest=max(lens))
    need = [-(-n // bs) for n in lens]
    s["block_table"], rest = _pages(case, need, max(need + [1]), g, B * width)
    s["dst_table"] = rest.view(B, width)
    s["cache"] = _random_cache(case, sum(need) + B * width, g)
    # a few keys hold most of the weight
    s["mass"] = torch.rand(sum(need) + B * width, Hkv, bs, generator=g, device="cuda").pow(8)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["keep"] = torch.full((B,), case["keep"], dtype=torch.int32, device="cuda")
    s["kept"] = torch.full((B, Hkv, case["keep"]), -1, dtype=torch.int32, device="cuda")
    s["out_lengths"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return _plan(s)


def _plan(s):
    """The scratch and the error word that a program keeps for the kernels."""
    if own:
        import speculative_decoding_pe_gb300 as pe
        c = s["case"]
        s["err"] = pe.new_error_word()
        if c["op"] == "verify":
            s["workspace"] = pe.new_filtered_workspace(c["B"], c["Kp"])
        elif c["op"] == "weigh":
            s["workspace"] = pe.new_weigh_workspace(*s["q"].shape[:2], s["block_table"].shape[1], c["bs"])
    return s


# -------------------------------------------------------------------- runs
def run(state):
    op = state["case"]["op"]
    if own:
        return {"sample": _own_sample, "verify": _own_verify, "weigh": _own_weigh, "evict": _own_evict}[op](state)
    return {"sample": _sample, "verify": _verify, "weigh": _weigh, "evict": _evict}[op](state)


def _own_sample(s):
    import speculative_decoding_pe_gb300 as pe
    pe.draft_sample(s["logits"], s["u"], s["tokens"], s["err"], out_prob=s["prob"], **s["asked"])
    return {"tokens": s["tokens"], "prob": s["prob"]}


def _own_verify(s):
    import speculative_decoding_pe_gb300 as pe
    pe.verify_filtered(s["target"], s["draft"], s["case"]["Kp"], s["tokens"], s["coins"], s["u"], s["accepted"], s["bonus"],
                       s["workspace"], s["err"], accept_prob=s["chance"], **s["asked"])
    return {"accepted": s["accepted"], "bonus": s["bonus"], "chance": s["chance"]}


def _own_weigh(s):
    import speculative_decoding_pe_gb300 as pe
    pe.kv_weigh(s["q"], s["cache"], s["block_table"], None, s["positions"], s["is_rejected"], s["mass"], s["out"],
                s["workspace"], s["err"], fresh=s["fresh"], scale=s["scale"])
    return {"mass": s["out"]}


def _own_evict(s):
    import speculative_decoding_pe_gb300 as pe
    c = s["case"]
    pe.kv_evict(s["cache"], s["mass"], s["block_table"], s["dst_table"], s["lengths"], s["keep"], s["kept"], s["out_lengths"],
                s["err"], sinks=c["sinks"], recent=c["recent"])
    return _evicted(s)


def _evicted(s):
    """The kept keys and, bit for bit, the pages that they went to."""
    return {"kept": s["kept"], "lengths": s["out_lengths"], "cache": s["cache"], "mass": s["mass"]}


# ------------------------------------------------------------- plain forms
def _kept_weights(logits, asked):
    """fp64 weights [n, V] of the kept columns, relative to the largest, zero elsewhere.  In 64 bits: a draw falls
    between the sums of up to V weights."""
    n, V = logits.shape
    t, k, p, m = (asked[a][:, None] for a in ("temperature", "top_k", "top_p", "min_p"))
    x, col = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    x = x.double()
    top = x[:, :1]
    w = torch.where(x == top, 1.0, ((x - top) / torch.where(t > 0, t, 1.0).double()).exp())
    rank = torch.arange(V, device=x.device)
    k = torch.where(t == 0, 1, torch.where(k > 0, k, V))
    w = torch.where(rank < k, w, 0.0)
    run = w.cumsum(1)
    w = torch.where((p >= 1) | (rank == 0) | (run - w < p.double() * run[:, -1:]), w, 0.0)
    w = torch.where((m <= 0) | (x >= top + torch.where(t > 0, t, 1.0).double() * m.double().clamp(min=1e-300, max=1.0).log()), w, 0.0)
    return torch.empty_like(w).scatter_(1, col, w)


def _drawn(w, u):
    """The first column whose running sum of weights exceeds u times the sum."""
    run = w.cumsum(1)
    return (run <= u.double()[:, None] * run[:, -1:]).sum(1).to(torch.int32)


def _sample(s):
    n = s["u"].numel()
    w = _kept_weights(s["logits"], {a: v.repeat_interleave(n // v.numel()) for a, v in s["asked"].items()})
    s["tokens"].copy_(_drawn(w, s["u"]))
    s["prob"].copy_(w.gather(1, s["tokens"][:, None].long())[:, 0] / w.sum(1))
    return {"tokens": s["tokens"], "prob": s["prob"]}


def _verify(s):
    B, Kp, V = s["case"]["B"], s["case"]["Kp"], s["case"]["V"]
    p = _kept_weights(s["target"], {a: v.repeat_interleave(Kp + 1) for a, v in s["asked"].items()})
    q = _kept_weights(s["draft"], {a: v.repeat_interleave(Kp) for a, v in s["asked"].items()})
    p = p.div_(p.sum(1, keepdim=True)).view(B, Kp + 1, V)
    q = q.div_(q.sum(1, keepdim=True)).view(B, Kp, V)
    x = s["tokens"].view(B, Kp + 1)[:, 1:, None].long()
    px, qx = p[:, :Kp].gather(2, x)[..., 0], q.gather(2, x)[..., 0]
    ok = s["coins"].view(B, Kp).double() * qx < px
    s["chance"].copy_(torch.where(px < qx, px / qx, torch.where(px > 0, 1.0, 0.0)).flatten())
    a = ok.int().cumprod(1).sum(1)
    b = torch.arange(B, device=a.device)
    pa = p[b, a]
    rest = (pa - q[b, a.clamp(max=Kp - 1)]).clamp_(min=0)
    rest = torch.where(((a < Kp) & (rest.sum(1) > 0))[:, None], rest, pa)
    s["accepted"].copy_(a)
    s["bonus"].copy_(_drawn(rest, s["u"]))
    return {"accepted": s["accepted"], "bonus": s["bonus"], "chance": s["chance"]}


def _keys(cache, D):
    """fp32 keys [..., 16, D] of records."""
    codes, scales = cache[..., :8 * D].unflatten(-1, (16, -1)), cache[..., 16 * D:17 * D].unflatten(-1, (16, -1))
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=cache.device)
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return (grid[both.int()].unflatten(-1, (-1, 16)) * scales.contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _weigh(s):
    c, bs, m = s["case"], s["case"]["bs"], s["m"]
    D, Hq, Hkv, B = c["D"], c["Hq"], c["Hkv"], c["B"]
    width = -(-s["longest"] // bs)
    limit = torch.where(s["is_rejected"] != 0, 0, s["positions"] + 1).view(B, m)
    t = torch.arange(width * bs, device=limit.device)
    step = max(1, (1 << 31) // (width * bs * max(m * Hq, 2 * Hkv * D)))
    for b in range(0, B, step):  # requests whose keys and scores fit some 8 GB each
        e = min(B, b + step)
        table = s["block_table"][b:e, :width].long()
        k = _keys(s["cache"][table], D)  # [g, width, Hkv, bs/16, 16, D]
        k = k.permute(0, 2, 1, 3, 4, 5).reshape(e - b, Hkv, -1, D)
        q = s["q"].view(B, m, Hkv, -1, D)[b:e].float().permute(0, 2, 1, 3, 4).reshape(e - b, Hkv, -1, D)
        z = (q * s["scale"]) @ k.transpose(2, 3)
        z.masked_fill_(~(t < limit[b:e].repeat_interleave(Hq // Hkv, 1)[:, None, :, None]), -math.inf)
        z.sub_(z.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
        total = z.sum(-1, keepdim=True)
        z.div_(torch.where(total > 0, total, 1.0))
        new = z.sum(2).view(e - b, Hkv, width, bs)
        seen = t < limit[b:e].amax(1)[:, None]
        old = torch.where(t < s["fresh"][b:e, None], 1.0, 0.0).view(e - b, 1, width, bs) * s["mass"][table].permute(0, 2, 1, 3)
        blk, off = table[:, t // bs][seen], (t % bs).expand(e - b, -1)[seen]
        s["out"][blk, :, off] = (new + old).flatten(2).permute(0, 2, 1)[seen]
    return {"mass": s["out"]}


def _evict(s):
    c, bs = s["case"], s["case"]["bs"]
    D, Hkv, B, keep = c["D"], c["Hkv"], c["B"], c["keep"]
    n, L = s["lengths"].long(), max(1, s["longest"])
    j = torch.arange(L, device=n.device)
    table = s["block_table"].long()
    mass = s["mass"][table[:, j // bs], :, j % bs].transpose(1, 2)  # [B, Hkv, L]
    size = torch.minimum(n, s["keep"].long())
    first = size.clamp(max=c["sinks"])
    last = torch.minimum(size - first, torch.full_like(size, c["recent"]))
    held = (j < first[:, None]) | (j >= (n - last)[:, None])
    mass = torch.where(held[:, None], math.inf, mass)
    mass = torch.where((j < n[:, None])[:, None], mass, -math.inf)
    order = torch.sort(mass, dim=2, descending=True, stable=True)[1][..., :keep]
    i = torch.arange(order.shape[2], device=n.device)
    order = torch.where(i < size[:, None, None], order, L).sort(2)[0]  # ascending, then what is not kept
    b, h, i = (order < L).nonzero(as_tuple=True)
    src = order[b, h, i]
    s["kept"][b, h, i] = src.to(torch.int32)
    s["out_lengths"].copy_(size)
    at = [(t[b, x // bs].long(), h, x % bs // 16, x % 16) for t, x in ((s["block_table"], src), (s["dst_table"], i))]
    for lo, hi in ((0, 8 * D), (8 * D, 16 * D), (16 * D, 17 * D), (17 * D, 18 * D)):  # the parts of a record
        part = s["cache"][..., lo:hi].unflatten(-1, (16, -1))
        part[at[1]] = part[at[0]]
    s["mass"][at[1][0], h, i % bs] = s["mass"][at[0][0], h, src % bs]
    return _evicted(s)


# -------------------------------------------------------------------- work
def work(case):
    B, op = case["B"], case["op"]
    if op == "sample":
        n = B * case["K"]
        return {"bytes": n * case["V"] * (4 if case["fp32"] else 2) + 12 * n + 16 * B, "flops": 4 * n * case["V"]}
    if op == "verify":
        n = B * (2 * case["Kp"] + 1)
        return {"bytes": n * case["V"] * (4 if case["fp32"] else 2) + 16 * n + 28 * B, "flops": 4 * n * case["V"]}
    Hkv, D, bs = case["Hkv"], case["D"], case["bs"]
    if op == "weigh":
        rows = _rows(case)
        seen = [[p + 1 if k else 0 for p, k in r] for r in rows]
        keys = sum(max(r) for r in seen)
        # each key's codes and scales, its mass read and written, the queries, the table
        return {"bytes": keys * Hkv * (D // 2 + D // 16 + 8) + len(rows) * len(rows[0]) * (2 * case["Hq"] * D + 5) + 4 * keys // bs,
                "flops": sum(map(sum, seen)) * case["Hq"] * (2 * D + 4)}
    lens = _lengths(case)
    kept = sum(min(n, case["keep"]) for n in lens)
    over = sum(n for n in lens if n > case["keep"])  # only these masses decide anything
    return {"bytes": Hkv * (4 * over + kept * (2 * (18 * D // 16) + 12)) + 4 * sum(-(-n // bs) for n in lens) + 12 * B,
            "flops": Hkv * over}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """From the definitions, in 64 bits, one row or request after another."""
    if case["op"] == "evict":
        return None  # nothing is computed: keys and masses are moved
    w = work(case)
    if w["flops"] > (6e11 if case["op"] == "weigh" else 4e8):
        return None
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    return _exact_weigh(s) if case["op"] == "weigh" else _exact_verify(s)


def _exact_row(x, t, k, p, m):
    """Probabilities of one fp64 row under one request's filters."""
    V = x.numel()
    if t == 0:
        return torch.nn.functional.one_hot(x.argmax(), V).double()
    z = torch.softmax(x / t, 0)
    value, col = z.sort(descending=True, stable=True)
    n = min(k, V) if k > 0 else V
    if p < 1:
        n = min(n, 1 + int((value[:n].cumsum(0)[:-1] < p * value[:n].sum()).sum()))
    if m > 0:
        n = min(n, int((value >= value[0] * m).sum()))
    out = torch.zeros_like(z)
    out[col[:n]] = value[:n] / value[:n].sum()
    return out


def _exact_draw(z, u):
    return int(torch.searchsorted(z.cumsum(0), u * z.sum(), right=True).clamp(max=z.numel() - 1))


def _exact_sample(s):
    K = s["case"]["K"]
    asked = [v.tolist() for v in s["asked"].values()]
    tokens, prob = [], []
    for i, u in enumerate(s["u"].tolist()):
        z = _exact_row(s["logits"][i].double(), *(v[i // K] for v in asked))
        tokens.append(_exact_draw(z, u))
        prob.append(float(z[tokens[-1]]))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "prob": torch.tensor(prob, dtype=torch.float64)}


def _exact_verify(s):
    Kp = s["case"]["Kp"]
    asked = [v.tolist() for v in s["asked"].values()]
    tokens, coins = s["tokens"].tolist(), s["coins"].tolist()
    accepted, bonus, chance = [], [], []
    for b, u in enumerate(s["u"].tolist()):
        a, rest = Kp, _exact_row(s["target"][b * (Kp + 1) + Kp].double(), *(v[b] for v in asked))
        for j in reversed(range(Kp)):  # the first rejection decides last
            x = tokens[b * (Kp + 1) + j + 1]
            z, q = (_exact_row(r.double(), *(v[b] for v in asked)) for r in (s["target"][b * (Kp + 1) + j], s["draft"][b * Kp + j]))
            px, qx = float(z[x]), float(q[x])
            chance.append(px / qx if px < qx else float(px > 0))
            if not coins[b * Kp + j] * qx < px:
                a, rest = j, (z - q).clamp(min=0)
                rest = rest if float(rest.sum()) > 0 else z
        chance[-Kp:] = chance[-Kp:][::-1]
        accepted.append(a)
        bonus.append(_exact_draw(rest, u))
    return {"accepted": torch.tensor(accepted, dtype=torch.int32), "bonus": torch.tensor(bonus, dtype=torch.int32),
            "chance": torch.tensor(chance, dtype=torch.float64)}


def _exact_weigh(s):
    c, m, bs = s["case"], s["m"], s["case"]["bs"]
    D, G = c["D"], c["Hq"] // c["Hkv"]
    signed = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device="cuda")
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    e = torch.arange(D, device="cuda")
    for b in range(c["B"]):
        r = slice(b * m, b * m + m)
        sees = (s["positions"][r].long() + 1) * (s["is_rejected"][r] == 0)
        L = int(sees.max())
        t = torch.arange(L, device="cuda")
        blk = s["block_table"][b].long()[t // bs]
        for h in range(c["Hkv"]):
            rec = s["cache"][blk, h, t % bs // 16]
            byte = rec.gather(1, (t % 16)[:, None] * (D // 2) + e // 2).int()
            sc = rec.gather(1, 16 * D + (t % 16)[:, None] * (D // 16) + e // 16).contiguous()
            k = signed[(byte >> (4 * (e % 2))) & 15] * sc.view(torch.float8_e4m3fn).double()
            z = torch.einsum("mgd,ld->mgl", s["q"][r, h * G:(h + 1) * G].double(), k) * s["scale"]
            z = z.masked_fill(t >= sees[:, None, None], -math.inf)
            z = torch.softmax(z, -1).nan_to_num(0.0).sum((0, 1))
            out[blk, h, t % bs] = z + torch.where(t < s["fresh"][b], s["mass"][blk, h, t % bs].double(), 0.0)
    return {"mass": out}
