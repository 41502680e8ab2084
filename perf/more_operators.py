"""Timing cases of latent attention served from a paged cache.

In latent attention all heads of a token share one latent vector and one rotated
key part, which is all that the cache holds.  Four operators, used together in a
serving step: a step's latent vectors are normalised and written with their
rotated keys, while the queries' rotary part is rotated as well (``append``);
single tokens attend over the cached rows themselves, the key's expansion being
folded into the query (``latent``); prompt chunks read the cached rows back in
order (``gather``), expand them to keys and values of every head with a product
of the model's, and attend over those (``expanded``).

``run`` computes an operator in its plain form with elementary torch operations,
or, with ``own`` set, through the library's entry points.  ``exact`` restates
each operator in 64 bits, apart from the plain form.
"""

import math

import numpy as np
import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
BS = 16                                   # tokens per cache block
ROPE = 64                                 # rotated dimensions of a key or a query head
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 64 requests: latency counts
        dict(name="append-decode-64", op="append", dtype="bf16", tokens=64, heads=32, nope=128,
             latent=512, interleaved=True, norm=True),
        # prompts of 16384 tokens in all
        dict(name="append-prompts-16384", op="append", dtype="bf16", tokens=16384, heads=32,
             nope=128, latent=512, interleaved=False, norm=True),
        # the contexts of a step's prompt chunks under a 2048-token budget
        dict(name="gather-chunks-4", op="gather", dtype="bf16", seqs=4, lo=512, hi=4096,
             latent=512),
        # four long contexts
        dict(name="gather-4x32k", op="gather", dtype="bf16", seqs=4, lo=32000, hi=32768,
             latent=512),
        # single precision, few heads, a short latent vector: the smallest attention call
        dict(name="latent-f32-8", op="latent", dtype="f32", seqs=8, qlen=1, heads=8, latent=256,
             lo=128, hi=2048),
        # four requests of 32k tokens: few rows, long contexts, latency counts
        dict(name="latent-4x32k", op="latent", dtype="bf16", seqs=4, qlen=1, heads=64, latent=512,
             lo=32000, hi=32768),
        # the ordinary decode batch: 64 requests of 512 to 4096 tokens
        dict(name="latent-64x4k", op="latent", dtype="bf16", seqs=64, qlen=1, heads=32, latent=512,
             lo=512, hi=4096),
        # a large decode batch of a model with many heads
        dict(name="latent-96x8k-h128", op="latent", dtype="bf16", seqs=96, qlen=1, heads=128,
             latent=512, lo=1024, hi=8192),
        # three speculated tokens a request are checked at once, a head count of 24
        dict(name="latent-32x8k-q3", op="latent", dtype="bf16", seqs=32, qlen=3, heads=24,
             latent=512, lo=1024, hi=8192),
        # single precision, small heads, ragged short prompts
        dict(name="expanded-f32-6", op="expanded", dtype="f32", seqs=6, heads=4, dim=64, q_lo=1,
             q_hi=300, c_lo=0, c_hi=200),
        # a 2048-token step: four prompt chunks of up to 512 tokens over cached prefixes
        dict(name="expanded-chunks-4", op="expanded", dtype="bf16", seqs=4, heads=32, dim=128,
             q_lo=400, q_hi=512, c_lo=512, c_hi=3584),
        # prompts of up to 4096 tokens, ragged
        dict(name="expanded-prompts-8", op="expanded", dtype="bf16", seqs=8, heads=32, dim=128,
             q_lo=1700, q_hi=4096, c_lo=0, c_hi=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "gather", "latent", "latent", "expanded"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    es = 4 if dtype == "f32" else 2
    latent = rng.choice([128, 256, 384, 512, 512])
    if op == "append":
        heads = rng.randint(1, 64)
        tokens = min(_log_int(rng, 1, 16384), 16384 * 32 * 2 // (heads * es))
        return dict(op=op, dtype=dtype, tokens=tokens, heads=heads, nope=rng.choice([0, 64, 128]),
                    latent=latent, interleaved=rng.random() < 0.5, norm=rng.random() < 0.7)
    if op == "gather":
        lo, hi = sorted(_log_int(rng, 1, 32768) for _ in range(2))
        seqs = max(1, min(_log_int(rng, 1, 256), 4 * 32768 * 2 // (hi * es)))
        return dict(op=op, dtype=dtype, seqs=seqs, lo=lo, hi=hi, latent=latent)
    if op == "latent":
        heads = rng.randint(1, 128)
        qlen = rng.choice([1, 1, rng.randint(2, 4), rng.randint(5, 40)])
        lo = _log_int(rng, qlen, 16384)
        hi = _log_int(rng, max(lo, 256), 32768)
        # the single-precision form works on the ordinary cores: smaller cases of it
        most = (96 * 128 * 4608) // (16 if dtype == "f32" else 1)
        seqs = max(1, min(_log_int(rng, 1, 256), 2 * most // (qlen * heads * (lo + hi)),
                          96 * 8192 * 2 // (hi * es)))
        hi = max(lo, min(hi, 2 * most // (seqs * qlen * heads)))
        return dict(op=op, dtype=dtype, seqs=seqs, qlen=qlen, heads=heads, latent=latent, lo=lo,
                    hi=hi)
    heads, dim = rng.randint(1, 48), rng.choice([64, 128, 128])
    q_lo, q_hi = sorted(_log_int(rng, 1, 4096) for _ in range(2))
    c_lo, c_hi = sorted(_log_int(rng, 1, 4096) - 1 for _ in range(2))
    if rng.random() < 0.4:
        c_lo = c_hi = 0
    most = (8 * 32 * 2900 * 2900) // (40 if dtype == "f32" else 1)
    q_hi = max(q_lo, min(q_hi, most // (heads * (q_hi + c_hi))))
    seqs = max(1, min(_log_int(rng, 1, 64), most // (heads * q_hi * (q_hi + c_hi)),
                      (1 << 19) // (heads * (q_hi + c_hi) // 8 + 1)))
    return dict(op=op, dtype=dtype, seqs=seqs, heads=heads, dim=dim, q_lo=q_lo, q_hi=q_hi,
                c_lo=c_lo, c_hi=c_hi)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _lens(gen, n, lo, hi):
    """n whole numbers of lo .. hi, drawn on the host."""
    return torch.randint(lo, hi + 1, (n,), generator=gen)


def _spread(gen, n, lo, hi):
    """n whole numbers evenly over lo .. hi in an order drawn on the host: their sum, and
    with it the outputs' shape, is the case's."""
    at = torch.arange(n, dtype=torch.float64) / max(1, n - 1) if n > 1 else torch.tensor([0.5])
    return (lo + (hi - lo) * at).round().long()[torch.randperm(n, generator=gen)]


def _ceil_blocks(x):
    return (x + BS - 1) // BS


def _dev(x):
    return x.to(torch.int32).to(DEVICE)


def _starts(lens):
    return torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])


def _randn(seed, shape, dtype, scale=1.0):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)
    return x.mul_(scale) if scale != 1.0 else x


def _block_tables(gen, lens):
    """Tables over a shuffled pool 5 % larger than needed, -1 behind a row's blocks."""
    blocks = _ceil_blocks(lens)
    total = int(blocks.sum())
    pool = total + max(4, total // 20)
    ids = torch.randperm(pool, generator=gen)
    width = max(1, int(blocks.max()))
    tables = torch.full((lens.numel(), width), -1, dtype=torch.int64)
    tables[torch.arange(width)[None, :] < blocks[:, None]] = ids[:total]
    return tables, pool


def rotary_table(positions, dim=ROPE, base=10000.0):
    """[positions][dim] fp32: cosines of a position's dim / 2 angles, then their sines."""
    inv = base ** (-np.arange(dim // 2, dtype=np.float64) * 2.0 / dim)
    ang = np.arange(positions, dtype=np.float64)[:, None] * inv[None, :]
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def _prepare_append(case, gen, seed):
    n, dt, rank = case["tokens"], DTYPES[case["dtype"]], case["latent"]
    pool = _ceil_blocks(n) + 4 + n // 64
    slots = torch.randperm(pool * BS, generator=gen)[:n]
    positions = _lens(gen, n, 0, 8191)
    # what the model's projections leave: latent and rotary key side by side, and
    # queries whose rotary part is the end of each head
    down = _randn(seed, (n, rank + ROPE), dt)
    q = _randn(seed + 1, (n, case["heads"], case["nope"] + ROPE), dt)
    return dict(op="append", down=down, q=q, rank=rank, heads=case["heads"], nope=case["nope"],
                interleaved=case["interleaved"],
                weight=_randn(seed + 2, (rank,), dt, 0.1).add_(1.0) if case["norm"] else None,
                slots=slots.to(DEVICE), positions=_dev(positions),
                table=torch.from_numpy(rotary_table(8192)).to(DEVICE),
                cache=torch.zeros((pool, BS, rank + ROPE), dtype=dt, device=DEVICE),
                # the absorbed queries' buffer: the rotated part is its last columns
                absorbed=torch.zeros((n, case["heads"], rank + ROPE), dtype=dt, device=DEVICE))


def _prepare_gather(case, gen, seed):
    lens = _spread(gen, case["seqs"], case["lo"], case["hi"])
    tables, pool = _block_tables(gen, lens)
    dt, rank, n = DTYPES[case["dtype"]], case["latent"], int(lens.sum())
    return dict(op="gather", rank=rank, tables=_dev(tables), starts=_dev(_starts(lens)),
                cache=_randn(seed, (pool, BS, rank + ROPE), dt),
                latent=torch.empty((n, rank), dtype=dt, device=DEVICE),
                rope=torch.empty((n, ROPE), dtype=dt, device=DEVICE))


def _prepare_latent(case, gen, seed):
    n, qlen, rank = case["seqs"], case["qlen"], case["latent"]
    lo, hi = max(case["lo"], qlen), max(case["hi"], qlen)
    lens = _lens(gen, n, lo, hi)
    tables, pool = _block_tables(gen, lens)
    dt = DTYPES[case["dtype"]]
    q = _randn(seed + 1, (n * qlen, case["heads"], rank + ROPE), dt)
    return dict(op="latent", rank=rank, heads=case["heads"], qlen=qlen, tables=_dev(tables),
                ctx=_dev(lens), most=hi, starts=_dev(torch.arange(n + 1) * qlen),
                cache=_randn(seed, (pool, BS, rank + ROPE), dt), q=q,
                scale=1.0 / math.sqrt(128 + ROPE),
                out=torch.empty((n * qlen, case["heads"], rank), dtype=dt, device=DEVICE))


def _prepare_expanded(case, gen, seed):
    new = _spread(gen, case["seqs"], case["q_lo"], case["q_hi"])
    keys = new + _spread(gen, case["seqs"], case["c_lo"], case["c_hi"])
    dt, h, d = DTYPES[case["dtype"]], case["heads"], case["dim"]
    nq, nk = int(new.sum()), int(keys.sum())
    # the expansion product leaves each head's key and value side by side
    kv = _randn(seed, (nk, h, 2 * d), dt)
    return dict(op="expanded", heads=h, dim=d, kv=kv, k=kv[..., :d], v=kv[..., d:],
                k_rope=_randn(seed + 1, (nk, ROPE), dt),
                q=_randn(seed + 2, (nq, h, d + ROPE), dt), q_starts=_dev(_starts(new)),
                k_starts=_dev(_starts(keys)), most=int(new.max()),
                host=(new.tolist(), keys.tolist()), scale=1.0 / math.sqrt(d + ROPE),
                out=torch.empty((nq, h, d), dtype=dt, device=DEVICE))


def prepare(case, seed):
    gen = torch.Generator()
    gen.manual_seed(seed)
    return {"append": _prepare_append, "gather": _prepare_gather, "latent": _prepare_latent,
            "expanded": _prepare_expanded}[case["op"]](case, gen, 7919 * seed)


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def _plain_rotate(x, cos, sin, interleaved):
    """x [..., 64] in single precision."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)


def _plain_append(s):
    rank, dt = s["rank"], s["cache"].dtype
    x = s["down"][:, :rank].float()
    if s["weight"] is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    cs = s["table"][s["positions"].long()]
    cos, sin = cs[:, :ROPE // 2], cs[:, ROPE // 2:]
    key = _plain_rotate(s["down"][:, rank:].float(), cos, sin, s["interleaved"])
    rows = s["cache"].view(-1, rank + ROPE)
    rows[s["slots"]] = torch.cat([x, key], dim=-1).to(dt)
    q = _plain_rotate(s["q"][..., s["nope"]:].float(), cos[:, None], sin[:, None], s["interleaved"])
    s["absorbed"][..., rank:] = q.to(dt)
    return dict(cache=s["cache"], q=s["absorbed"][..., rank:])


def _plain_gather(s):
    start = s["starts"].long()
    t = torch.arange(s["latent"].shape[0], device=start.device)
    seq = torch.searchsorted(start[1:], t, right=True)
    pos = t - start[seq]
    rows = s["cache"][s["tables"].long()[seq, pos // BS], pos % BS]
    return dict(latent=rows[:, :s["rank"]].contiguous(), rope=rows[:, s["rank"]:].contiguous())


def _plain_latent(s):
    n, qlen, rank, h = s["ctx"].numel(), s["qlen"], s["rank"], s["heads"]
    ctx, out = s["ctx"].long(), torch.empty_like(s["out"])
    width = s["tables"].shape[1]
    # a few sequences at a time: their rows in single precision stay below 4 GB
    group = max(1, (1 << 30) // (width * BS * (rank + ROPE)))
    group = max(1, min(group, (1 << 30) // (width * BS * qlen * h)))
    for a in range(0, n, group):
        b = min(n, a + group)
        rows = s["cache"][s["tables"][a:b].long().clamp(min=0)].flatten(1, 2).float()
        q = s["q"][a * qlen:b * qlen].float().view(b - a, qlen * h, rank + ROPE)
        x = (q @ rows.transpose(1, 2)) * s["scale"]
        last = ctx[a:b, None] - qlen + torch.arange(qlen, device=ctx.device)[None, :]
        key = torch.arange(width * BS, device=ctx.device)
        seen = (key[None, None, :] <= last[:, :, None])[:, :, None, :].expand(-1, -1, h, -1)
        x = torch.where(seen.reshape(x.shape), x, -math.inf)
        p = torch.exp(x - x.amax(-1, keepdim=True))
        o = (p @ rows[..., :rank]) / p.sum(-1, keepdim=True)
        out[a * qlen:b * qlen] = o.view(-1, h, rank).to(out.dtype)
    return out


def _plain_expanded(s):
    out, h, d = torch.empty_like(s["out"]), s["heads"], s["dim"]
    new, keys = s["host"]
    q0 = k0 = 0
    for m, n in zip(new, keys):
        q = s["q"][q0:q0 + m].float().transpose(0, 1)
        k = torch.cat([s["k"][k0:k0 + n].float(),
                       s["k_rope"][k0:k0 + n, None].float().expand(-1, h, -1)], -1).transpose(0, 1)
        v = s["v"][k0:k0 + n].float().transpose(0, 1)
        last = n - m + torch.arange(m, device=q.device)
        seen = torch.arange(n, device=q.device)[None, :] <= last[:, None]
        x = torch.where(seen, (q @ k.transpose(1, 2)) * s["scale"], -math.inf)
        p = torch.exp(x - x.amax(-1, keepdim=True))
        o = (p @ v) / p.sum(-1, keepdim=True)
        out[q0:q0 + m] = o.transpose(0, 1).to(out.dtype)
        q0, k0 = q0 + m, k0 + n
    return out


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _handle(s, pkv):
    """What a program keeps between calls: the descriptor and the workspace."""
    if "handle" not in s:
        s["handle"] = pkv.latent_desc(s["cache"], s["rank"], s.get("heads", 1))
        if s["op"] == "latent":
            s["ws"] = pkv.workspace(pkv.latent_workspace_bytes(
                s["handle"], s["ctx"].numel(), s["q"].shape[0], s["most"]))
    return s["handle"]


def run(state):
    s = state
    if not own:
        return {"append": _plain_append, "gather": _plain_gather, "latent": _plain_latent,
                "expanded": _plain_expanded}[s["op"]](s)
    import paged_kv_cache_51_gb300 as pkv

    if s["op"] == "expanded":
        return pkv.pkv_attention_expanded(s["out"], s["q"], s["k"], s["v"], s["k_rope"],
                                          s["q_starts"], s["k_starts"], s["most"], s["scale"])
    h, rank = _handle(s, pkv), s["rank"]
    if s["op"] == "append":
        rotated = s["absorbed"][..., rank:]
        pkv.paged_latent_append(s["down"][:, :rank], s["down"][:, rank:], s["slots"],
                                s["positions"], s["table"], s["cache"], h,
                                norm_weight=s["weight"], eps=EPS, q=s["q"][..., s["nope"]:],
                                q_out=rotated, interleaved=s["interleaved"])
        return dict(cache=s["cache"], q=rotated)
    if s["op"] == "gather":
        pkv.paged_latent_gather(s["latent"], s["rope"], s["cache"], h, s["tables"], s["starts"])
        return dict(latent=s["latent"], rope=s["rope"])
    return pkv.paged_attention_latent(s["out"], s["q"], s["cache"], h, s["tables"], s["ctx"],
                                      s["most"], s["scale"],
                                      query_start_loc=s["starts"] if s["qlen"] > 1 else None,
                                      ws=s["ws"])


# ----------------------------------------------------------------------------
# what a pass cannot do without (expected values over the lengths' ranges)
# ----------------------------------------------------------------------------
def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "append":
        n, h, rank = case["tokens"], case["heads"], case["latent"]
        # a position's cosines and sines are 64 values, read once for each token
        return dict(bytes=n * (2 * (rank + ROPE) * es + 2 * h * ROPE * es + 4 * ROPE + 12)
                    + rank * es, flops=n * (4 * rank + 3 * ROPE * (h + 1)))
    if case["op"] == "gather":
        n = case["seqs"] * (case["lo"] + case["hi"]) / 2
        return dict(bytes=n * 2 * (case["latent"] + ROPE) * es + 4 * n / BS, flops=0)
    if case["op"] == "latent":
        n, qlen, h, rank = case["seqs"], case["qlen"], case["heads"], case["latent"]
        mean = (max(case["lo"], qlen) + max(case["hi"], qlen)) / 2
        return dict(bytes=n * (mean * (rank + ROPE) * es + 4 * mean / BS + 4
                               + qlen * h * (2 * rank + ROPE) * es),
                    flops=2 * n * qlen * (mean - (qlen - 1) / 2) * h * (2 * rank + ROPE))
    h, d = case["heads"], case["dim"]
    qs = [case["q_lo"], (case["q_lo"] + case["q_hi"]) / 2, case["q_hi"]]
    mean_q = qs[1]
    # the mean of q^2 over a uniform range, and of the prefix
    mean_qq = (qs[0] ** 2 + 4 * qs[1] ** 2 + qs[2] ** 2) / 6
    mean_c = (case["c_lo"] + case["c_hi"]) / 2
    pairs = case["seqs"] * (mean_qq / 2 + mean_q / 2 + mean_q * mean_c)
    return dict(bytes=case["seqs"] * es * ((mean_q + mean_c) * (h * 2 * d + ROPE)
                                           + mean_q * h * (2 * d + ROPE)),
                flops=2 * pairs * h * (2 * d + ROPE))


# ----------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms
# ----------------------------------------------------------------------------
def _exact_rotate(x, angles_cos, angles_sin, interleaved):
    """Each pair (x_i, y_i) as a complex number times cos + i sin; NumPy, 64 bits."""
    half = x.shape[-1] // 2
    at = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, half),
                                                                     slice(half, None))
    z = (x[..., at[0]] + 1j * x[..., at[1]]) * (angles_cos + 1j * angles_sin)
    y = np.empty_like(x)
    y[..., at[0]], y[..., at[1]] = z.real, z.imag
    return y


def _exact_append(s):
    rank = s["rank"]
    down = s["down"].double().cpu().numpy()
    x = down[:, :rank]
    if s["weight"] is not None:
        norm = np.sqrt(np.einsum("td,td->t", x, x) / rank + EPS)
        x = x * s["weight"].double().cpu().numpy()[None, :] / norm[:, None]
    cs = s["table"].cpu().numpy().astype(np.float64)[s["positions"].cpu().numpy()]
    cos, sin = cs[:, :ROPE // 2], cs[:, ROPE // 2:]
    cache = np.zeros(tuple(s["cache"].shape))
    slots = s["slots"].cpu().numpy()
    cache[slots // BS, slots % BS, :rank] = x
    cache[slots // BS, slots % BS, rank:] = _exact_rotate(down[:, rank:], cos, sin,
                                                          s["interleaved"])
    q = _exact_rotate(s["q"][..., s["nope"]:].double().cpu().numpy(), cos[:, None], sin[:, None],
                      s["interleaved"])
    return dict(cache=torch.from_numpy(cache), q=torch.from_numpy(q))


def _exact_gather(s):
    parts, start, tables = [], s["starts"].tolist(), s["tables"].cpu()
    cache = s["cache"].cpu()
    for i in range(len(start) - 1):
        n = start[i + 1] - start[i]
        ids = tables[i, :-(-n // BS)].long()
        parts.append(cache[ids].reshape(-1, cache.shape[2])[:n])
    rows = torch.cat(parts).double()
    return dict(latent=rows[:, :s["rank"]].contiguous(), rope=rows[:, s["rank"]:].contiguous())


def _exact_latent(s):
    """Request by request over its own rows, 8192 scores' rows at a time."""
    rank, h, qlen = s["rank"], s["heads"], s["qlen"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    for i, c in enumerate(s["ctx"].tolist()):
        ids = s["tables"][i, :-(-c // BS)].long()
        rows = s["cache"][ids].reshape(-1, rank + ROPE)[:c].double()
        for t in range(qlen):
            r, n = i * qlen + t, c - qlen + t + 1
            x = torch.einsum("hd,kd->hk", s["q"][r].double(), rows[:n]) * s["scale"]
            out[r] = torch.softmax(x, -1) @ rows[:n, :rank]
    return out


def _exact_expanded(s):
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    new, keys = s["host"]
    d, q0, k0 = s["dim"], 0, 0
    for m, n in zip(new, keys):
        shared = s["k_rope"][k0:k0 + n].double()
        hidden = torch.triu(torch.ones(m, n, dtype=torch.bool, device=out.device), n - m + 1)
        for h in range(s["heads"]):
            q = s["q"][q0:q0 + m, h].double()
            x = q[:, :d] @ s["k"][k0:k0 + n, h].double().t() + q[:, d:] @ shared.t()
            x = (x * s["scale"]).masked_fill_(hidden, -math.inf)
            out[q0:q0 + m, h] = torch.softmax(x, -1) @ s["v"][k0:k0 + n, h].double()
        q0, k0 = q0 + m, k0 + n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "gather": _exact_gather, "latent": _exact_latent,
            "expanded": _exact_expanded}[case["op"]](s)
