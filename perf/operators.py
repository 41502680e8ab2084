"""Timing cases of the operators for long contexts served from the device.

Four operators, used one after the other in a serving step that never returns to
the host: block tables and slots are built on the GPU from the requests'
lengths (``tables``), the key bounds of the blocks written in the step are
brought up to date (``bounds``), each query picks the blocks of its sequence
that a cheap score ranks highest (``select``), and attention reads those blocks
only (``attend``).

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
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one decode step of the Llama-2-7B batch: 64 requests, 512 to 4096 tokens
        dict(name="tables-decode-64", op="tables", seqs=64, chunks=0, chunk=1, lo=512, hi=4096),
        # a mixed step under a 2048-token budget: 512 decode rows, three prompt chunks
        dict(name="tables-mixed-2048", op="tables", seqs=515, chunks=3, chunk=512, lo=512, hi=3584),
        # a large decode batch of long contexts: wide tables
        dict(name="tables-decode-1024", op="tables", seqs=1024, chunks=0, chunk=1, lo=1024,
             hi=32768),
        # the open blocks of a decode step, one key/value head for each query head
        dict(name="bounds-decode-64", op="bounds", dtype="bf16", seqs=64, kv_heads=32, head_dim=128,
             new_lo=1, new_hi=1, lo=512, hi=4096),
        # prompts of 16384 tokens in all, ragged, grouped-query heads
        dict(name="bounds-prompts-16384", op="bounds", dtype="bf16", seqs=8, kv_heads=8,
             head_dim=128, new_lo=1700, new_hi=2048, lo=0, hi=700),
        # four requests of 32k tokens, groups of 8 query heads: few rows, long lists
        dict(name="select-4x32k", op="select", dtype="bf16", seqs=4, qlen=1, q_heads=64,
             kv_heads=8, head_dim=128, lo=32000, hi=32768, top_k=128, sink=1, recent=4),
        # the Llama-3-8B decode batch: 256 requests, 1k to 8k tokens
        dict(name="select-256x8k", op="select", dtype="bf16", seqs=256, qlen=1, q_heads=32,
             kv_heads=8, head_dim=128, lo=1024, hi=8192, top_k=64, sink=1, recent=2),
        # a full batch of long contexts, two query tokens a request (speculated tokens checked)
        dict(name="select-48x32k-q2", op="select", dtype="bf16", seqs=48, qlen=2, q_heads=32,
             kv_heads=8, head_dim=128, lo=8192, hi=32768, top_k=128, sink=1, recent=4),
        # single-precision caches, small heads: the smallest attention call
        dict(name="attend-f32-8", op="attend", dtype="f32", seqs=8, qlen=1, q_heads=8, kv_heads=8,
             head_dim=64, lo=128, hi=2048, top_k=16, sink=1, recent=1),
        # four requests of 32k tokens, groups of 8: few rows, latency counts
        dict(name="attend-4x32k", op="attend", dtype="bf16", seqs=4, qlen=1, q_heads=64,
             kv_heads=8, head_dim=128, lo=32000, hi=32768, top_k=128, sink=1, recent=4),
        # the Llama-3-8B decode batch over 64 blocks (1024 tokens) a head
        dict(name="attend-256x8k", op="attend", dtype="bf16", seqs=256, qlen=1, q_heads=32,
             kv_heads=8, head_dim=128, lo=1024, hi=8192, top_k=64, sink=1, recent=2),
        # the Llama-2-7B batch: 32 key/value heads, each with a list of its own
        dict(name="attend-64x4k-mha", op="attend", dtype="bf16", seqs=64, qlen=1, q_heads=32,
             kv_heads=32, head_dim=128, lo=2048, hi=4096, top_k=100, sink=2, recent=3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "bounds", "select", "attend"])
    if op == "tables":
        lo, hi = _log_int(rng, 1, 32768), _log_int(rng, 256, 32768)
        lo, hi = min(lo, hi), max(lo, hi)
        seqs = _log_int(rng, 1, 1024)
        chunks = rng.choice([0, 0, rng.randint(1, min(seqs, 8))])
        return dict(op=op, seqs=seqs, chunks=chunks,
                    chunk=_log_int(rng, 2, 2048) if chunks else 1, lo=lo, hi=hi)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
    d = rng.choice([64, 128, 128])
    if op == "bounds":
        new_lo, new_hi = sorted((_log_int(rng, 1, 2048), _log_int(rng, 1, 2048)))
        if rng.random() < 0.4:
            new_lo = new_hi = 1
        seqs = max(1, min(_log_int(rng, 1, 256), 16384 * 8 * 2 // (new_hi * kv * 4)))
        lo, hi = sorted(_log_int(rng, 1, 4096) for _ in range(2))
        return dict(op=op, dtype=dtype, seqs=seqs, kv_heads=kv, head_dim=d, new_lo=new_lo,
                    new_hi=new_hi, lo=lo, hi=hi)
    g = rng.choice([1, 2, 4, 8])
    kv = min(kv, 64 // g)
    qlen = rng.choice([1, 1, 1, rng.randint(2, 4)])
    sink, recent = rng.randint(0, 4), rng.randint(1, 6)
    # contexts from a token up to lengths of which a list leaves blocks out
    top_k = max(sink + recent, _log_int(rng, 1, 256))
    if op == "select":
        top_k = sink + recent + _log_int(rng, 2, 246)
    lo = _log_int(rng, qlen, 16384)
    hi = _log_int(rng, max(lo, 1024), 32768)
    most = 64 * 32 * 100 if op == "attend" else 96 * 8 * 1024
    each = qlen * kv * (top_k * (2 if dtype == "f32" else 1) if op == "attend" else -(-hi // BS))
    # caches of the attention cases stay below 8 GB
    room = (1 << 33) // (4 * hi * kv * d * 2) if op == "attend" else 1 << 20
    seqs = max(1, min(_log_int(rng, 1, 256), most // max(1, each), room))
    return dict(op=op, dtype=dtype, seqs=seqs, qlen=qlen, q_heads=kv * g, kv_heads=kv, head_dim=d,
                lo=lo, hi=hi, top_k=top_k, sink=sink, recent=recent)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _lens(gen, n, lo, hi):
    """n whole numbers of lo .. hi (at least 0), drawn on the host."""
    return torch.randint(lo, hi + 1, (n,), generator=gen)


def _block_tables(gen, blocks, width, pool=None):
    """Tables [n][width] over a shuffled pool (5 % larger than needed, unless its
    size is given), -1 behind each row's blocks; the pool's size and the shuffled
    ids that no row took."""
    total = int(blocks.sum())
    pool = total + max(4, total // 20) if pool is None else pool
    ids = torch.randperm(pool, generator=gen)
    tables = torch.full((blocks.numel(), width), -1, dtype=torch.int64)
    tables[torch.arange(width)[None, :] < blocks[:, None]] = ids[:total]
    return tables, pool, ids[total:]


def _ceil_blocks(x):
    return (x + BS - 1) // BS


def _prepare_tables(case, gen):
    n = case["seqs"]
    cached = _lens(gen, n, case["lo"], case["hi"])
    new = torch.ones(n, dtype=torch.int64)
    if case["chunks"]:
        at = torch.randperm(n, generator=gen)[:case["chunks"]]
        new[at] = _lens(gen, case["chunks"], max(1, case["chunk"] // 2), case["chunk"])
    width = -(-(case["hi"] + case["chunk"]) // BS)
    rows = n + max(1, n // 8)                  # rows of other, waiting requests among them
    seq_rows = torch.randperm(rows, generator=gen)[:n]
    need = int((_ceil_blocks(cached + new) - _ceil_blocks(cached)).sum())
    held, pool, rest = _block_tables(gen, _ceil_blocks(cached), width)
    more = torch.arange(pool, pool + need)     # room for the step's blocks
    pool += need
    table = torch.full((rows, width), -1, dtype=torch.int64)
    table[seq_rows] = held
    free = torch.cat([rest, more])
    free = free[torch.randperm(free.numel(), generator=gen)]
    stack = torch.zeros(pool, dtype=torch.int64)
    stack[:free.numel()] = free
    tokens = (n - case["chunks"]) + case["chunks"] * case["chunk"]

    def dev(x):
        return x.to(torch.int32).to(DEVICE)

    def out(*shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype, device=DEVICE)

    return dict(op="tables", table=dev(table), free_list=dev(stack),
                free_count=dev(torch.tensor([free.numel()])), seq_rows=dev(seq_rows),
                cached_lens=dev(cached), new_lens=dev(new), block_tables=out(n, width),
                context_lens=out(n), query_start_loc=out(n + 1),
                slot_mapping=out(tokens, dtype=torch.int64), positions=out(tokens),
                free_count_out=out(1))


def _randn(seed, shape, dtype, scale=1.0):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)
    return x.mul_(scale) if scale != 1.0 else x


def _prepare_bounds(case, gen, seed):
    n = case["seqs"]
    new = _lens(gen, n, case["new_lo"], case["new_hi"])
    ctx = _lens(gen, n, case["lo"], case["hi"]) + new
    # only the blocks that the step touches are laid out for real; the others are one block
    first, last = (ctx - new) // BS, (ctx - 1) // BS
    width = int(last.max()) + 1
    touched, pool, _ = _block_tables(gen, last - first + 1, int((last - first).max()) + 1,
                                     n * (case["new_hi"] // BS + 2))
    tables = torch.zeros((n, width), dtype=torch.int64)
    j = torch.arange(touched.shape[1])[None, :]
    have = j < (last - first + 1)[:, None]
    seq = torch.arange(n)[:, None].expand_as(have)
    tables[seq[have], (first[:, None] + j)[have]] = touched[have]
    k = _randn(seed, (pool, case["kv_heads"], BS, case["head_dim"]), DTYPES[case["dtype"]], 0.5)
    k *= _randn(seed + 1, (1, case["kv_heads"], 1, case["head_dim"]), torch.float32, 0.5).exp().to(
        k.dtype)                               # channels differ in size
    start = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
    return dict(op="bounds", k_cache=k, block_tables=tables.to(torch.int32).to(DEVICE),
                context_lens=ctx.to(torch.int32).to(DEVICE),
                query_start_loc=start.to(torch.int32).to(DEVICE), tokens=int(new.sum()),
                most=int((last - first).max()) + 1,
                bounds=torch.zeros((pool, case["kv_heads"], 2, case["head_dim"]),
                                   dtype=torch.int8, device=DEVICE),
                exps=torch.zeros((pool, case["kv_heads"]), dtype=torch.int8, device=DEVICE))


def _rows(case, gen):
    """Contexts, tables and the rows' visible keys of a select or attend case."""
    n, qlen = case["seqs"], case["qlen"]
    ctx = _lens(gen, n, max(case["lo"], qlen), max(case["hi"], qlen))
    blocks = _ceil_blocks(ctx)
    tables, pool, _ = _block_tables(gen, blocks, int(blocks.max()))
    row_seq = torch.arange(n).repeat_interleave(qlen)
    row_keys = (ctx[:, None] - qlen + 1 + torch.arange(qlen)[None, :]).reshape(-1)
    s = dict(op=case["op"], block_tables=tables.to(torch.int32).to(DEVICE),
             context_lens=ctx.to(torch.int32).to(DEVICE), max_context_len=max(case["hi"], qlen),
             query_start_loc=(torch.arange(n + 1) * qlen).to(torch.int32).to(DEVICE),
             qlen=qlen, q_heads=case["q_heads"], kv_heads=case["kv_heads"],
             head_dim=case["head_dim"], pool=pool)
    return s, pool, row_seq.to(DEVICE), row_keys.to(DEVICE)


def _prepare_select(case, gen, seed):
    s, pool, row_seq, row_keys = _rows(case, gen)
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed + 2)
    shape = (pool, case["kv_heads"], case["head_dim"])
    mid = torch.randn(shape, generator=g, device=DEVICE) * 25.0
    half = (torch.randn(shape, generator=g, device=DEVICE) * 8.0 + 30.0).abs()
    s["bounds"] = torch.stack([mid + half, mid - half], dim=2).clamp_(-127, 127).round_().to(
        torch.int8)
    s["exps"] = torch.randint(-7, -4, shape[:2], generator=g, device=DEVICE).to(torch.int8)
    rows = case["seqs"] * case["qlen"]
    s["q"] = _randn(seed, (rows, case["q_heads"], case["head_dim"]), DTYPES[case["dtype"]])
    s["selected"] = torch.empty((rows, case["kv_heads"], case["top_k"]), dtype=torch.int32,
                                device=DEVICE)
    s.update(top_k=case["top_k"], sink=case["sink"], recent=case["recent"], f32=case["dtype"] == "f32")
    return s


def _prepare_attend(case, gen, seed):
    s, pool, row_seq, row_keys = _rows(case, gen)
    dt = DTYPES[case["dtype"]]
    shape = (pool, case["kv_heads"], BS, case["head_dim"])
    s["k_cache"] = _randn(seed, shape, dt, 0.5)
    s["v_cache"] = _randn(seed + 1, shape, dt, 0.5)
    rows = case["seqs"] * case["qlen"]
    s["q"] = _randn(seed + 2, (rows, case["q_heads"], case["head_dim"]), dt)
    s["out"] = torch.empty_like(s["q"])
    # lists as a selection leaves them: the first and the last blocks, others
    # between, in ascending order, -1 behind a short list
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed + 3)
    width = s["block_tables"].shape[1]
    k = min(case["top_k"], width)
    blocks = _ceil_blocks(row_keys)[:, None, None]
    j = torch.arange(width, device=DEVICE)[None, None, :]
    want = torch.rand((rows, case["kv_heads"], width), generator=g, device=DEVICE)
    want = torch.where((j < case["sink"]) | (j >= blocks - case["recent"]), 2.0, want)
    want = torch.where(j < blocks, want, -1.0)
    val, idx = want.topk(k, dim=-1)
    idx = torch.where(val < 0, width, idx).sort(dim=-1).values
    idx = torch.where(idx == width, -1, idx)
    s["selected"] = torch.full((rows, case["kv_heads"], case["top_k"]), -1, dtype=torch.int32,
                               device=DEVICE)
    s["selected"][..., :k] = idx.to(torch.int32)
    return s


def prepare(case, seed):
    gen = torch.Generator()
    gen.manual_seed(seed)
    if case["op"] == "tables":
        return _prepare_tables(case, gen)
    return {"bounds": _prepare_bounds, "select": _prepare_select,
            "attend": _prepare_attend}[case["op"]](case, gen, 7919 * seed)


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def _plain_tables(s):
    rows, cached, new = s["seq_rows"].long(), s["cached_lens"].long(), s["new_lens"].long()
    table, width = s["table"], s["table"].shape[1]
    ctx = cached + new
    old, now = _ceil_blocks(cached), _ceil_blocks(ctx)
    taken = (now - old).cumsum(0)
    j = torch.arange(width, device=table.device)[None, :]
    # the k-th new block of the step is the k-th entry from the top of the stack
    at = s["free_count"].long() - 1 - ((taken - (now - old) - old)[:, None] + j)
    got = s["free_list"][at.clamp(0, s["free_list"].numel() - 1)]
    held = torch.where((j >= old[:, None]) & (j < now[:, None]), got, table[rows])
    table[rows] = held
    tables = torch.where(j < now[:, None], held, -1)
    start = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    t = torch.arange(s["slot_mapping"].numel(), device=table.device)
    live = t < start[-1]
    seq = torch.searchsorted(start[1:], t, right=True).clamp(max=rows.numel() - 1)
    pos = torch.where(live, cached[seq] + t - start[seq], 0)
    slots = tables[seq, pos // BS].long() * BS + pos % BS
    return dict(table=table, block_tables=tables, context_lens=ctx.int(),
                query_start_loc=start.int(), slot_mapping=torch.where(live, slots, -1),
                positions=pos.int(), free_count=s["free_count"] - taken[-1:].int())


def _exponent(amax):
    """The least e with amax <= 127 * 2^e, kept within -50 .. 50."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 127.0 / 128.0, x - 7, x - 6)
    return torch.where(amax > 0, e, torch.full_like(e, -50)).clamp(-50, 50)


def _plain_bounds(s):
    ctx, start = s["context_lens"].long(), s["query_start_loc"].long()
    first = (ctx - (start[1:] - start[:-1])) // BS
    block = first[:, None] + torch.arange(s["most"], device=ctx.device)[None, :]
    live = block <= ((ctx - 1) // BS)[:, None]
    phys = s["block_tables"].long().gather(1, block.clamp(max=s["block_tables"].shape[1] - 1))[live]
    rows = (ctx[:, None] - block * BS)[live].clamp(max=BS)
    k = s["k_cache"][phys].float()
    seen = (torch.arange(BS, device=ctx.device)[None, :] < rows[:, None])[:, None, :, None]
    hi = torch.where(seen, k, -math.inf).amax(2)
    lo = torch.where(seen, k, math.inf).amin(2)
    e = _exponent(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    unit = torch.ldexp(torch.ones_like(e, dtype=torch.float32), -e)[..., None]
    codes = torch.stack([(hi * unit).ceil(), (lo * unit).floor()], dim=2).clamp(-127, 127)
    s["bounds"][phys] = codes.to(torch.int8)
    s["exps"][phys] = e.to(torch.int8)
    return dict(bounds=s["bounds"], exps=s["exps"])


def _row_layout(s):
    rows = torch.arange(s["q"].shape[0], device=s["q"].device)
    seq = rows // s["qlen"]
    keys = s["context_lens"].long()[seq] - s["qlen"] + 1 + rows % s["qlen"]
    return seq, keys


def _plain_select(s):
    seq, keys = _row_layout(s)
    width, kv, d = s["block_tables"].shape[1], s["kv_heads"], s["head_dim"]
    g = s["q_heads"] // kv
    q = s["q"].float()
    eq = _exponent(q.abs().amax(-1))
    code = (q * torch.ldexp(torch.ones_like(eq, dtype=torch.float32), -eq)[..., None]).round()
    both = torch.cat([code.clamp(min=0), code.clamp(max=0)], -1).view(-1, kv, g, 2 * d)
    phys = s["block_tables"].long().clamp(min=0)
    ends = s["bounds"][phys].view(phys.shape[0], width, kv, 2 * d).permute(0, 2, 3, 1).float()
    if s["qlen"] == 1:
        dot = both @ ends                      # whole numbers below 2^24: exact
    else:
        dot = (both.view(-1, s["qlen"], kv, g, 2 * d) @ ends[:, None]).view(-1, kv, g, width)
    score = torch.ldexp(dot, eq.view(-1, kv, g)[..., None]).amax(2)
    score = torch.ldexp(score, s["exps"][phys].int().transpose(1, 2)[seq])
    blocks = _ceil_blocks(keys)[:, None, None]
    j = torch.arange(width, device=q.device)[None, None, :]
    score = torch.where((j < s["sink"]) | (j >= blocks - s["recent"]), math.inf, score)
    score = torch.where(j < blocks, score, -math.inf)
    k = min(s["top_k"], width)
    idx = score.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    idx = torch.where(idx < blocks, idx, width).sort(dim=-1).values
    s["selected"].fill_(-1)
    s["selected"][..., :k] = torch.where(idx == width, -1, idx).int()
    return s["selected"]


def _plain_attend(s):
    seq, keys = _row_layout(s)
    kv, d = s["kv_heads"], s["head_dim"]
    sel = s["selected"].long()
    phys = s["block_tables"].long()[seq[:, None, None], sel.clamp(min=0)].clamp(min=0)
    head = torch.arange(kv, device=sel.device)[None, :, None]
    q = s["q"].float().view(-1, kv, s["q_heads"] // kv, d)
    pos = sel[..., None] * BS + torch.arange(BS, device=sel.device)
    seen = ((sel[..., None] >= 0) & (pos < keys[:, None, None, None])).flatten(2)[:, :, None, :]
    k = s["k_cache"][phys, head].float().flatten(2, 3)
    score = torch.where(seen, q @ k.transpose(2, 3) * (1.0 / math.sqrt(d)), -math.inf)
    del k
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = p @ s["v_cache"][phys, head].float().flatten(2, 3) / p.sum(-1, keepdim=True)
    return o.view(s["q"].shape).to(s["q"].dtype)


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _handle(s, pkv):
    """What a program keeps between calls: the descriptor, the tables' handle and
    the selection's workspace."""
    if "handle" not in s:
        if s["op"] == "tables":
            s["handle"] = pkv.DeviceTables(s["table"], s["free_list"], s["free_count"], BS)
        elif s["op"] == "bounds":
            s["handle"] = pkv.cache_desc(s["k_cache"], s["k_cache"].shape[1])
        elif s["op"] == "attend":
            s["handle"] = pkv.cache_desc(s["k_cache"], s["q_heads"])
        else:
            s["handle"] = pkv.CacheDesc(pkv.PKV_F32 if s["f32"] else pkv.PKV_BF16, s["pool"], BS,
                                        s["kv_heads"], s["q_heads"], s["head_dim"])
            s["ws"] = pkv.workspace(pkv.select_workspace_bytes(
                s["handle"], s["q"].shape[0], s["max_context_len"]))
    return s["handle"]


def run(state):
    s = state
    if not own:
        return {"tables": _plain_tables, "bounds": _plain_bounds, "select": _plain_select,
                "attend": _plain_attend}[s["op"]](s)
    import paged_kv_cache_51_gb300 as pkv

    h = _handle(s, pkv)
    if s["op"] == "tables":
        pkv.pkv_tables_step(h, s["seq_rows"], s["cached_lens"], s["new_lens"], s["block_tables"],
                            s["context_lens"], s["query_start_loc"], s["slot_mapping"],
                            s["positions"], free_count_out=s["free_count_out"])
        return dict(table=s["table"], block_tables=s["block_tables"],
                    context_lens=s["context_lens"], query_start_loc=s["query_start_loc"],
                    slot_mapping=s["slot_mapping"], positions=s["positions"],
                    free_count=s["free_count_out"])
    if s["op"] == "bounds":
        pkv.pkv_block_bounds(s["bounds"], s["exps"], s["k_cache"], h, s["block_tables"],
                             s["context_lens"], query_start_loc=s["query_start_loc"],
                             num_query_tokens=s["tokens"])
        return dict(bounds=s["bounds"], exps=s["exps"])
    start = s["query_start_loc"] if s["qlen"] > 1 else None
    if s["op"] == "select":
        return pkv.pkv_select_blocks(s["selected"], s["q"], s["bounds"], s["exps"], h,
                                     s["block_tables"], s["context_lens"], s["max_context_len"],
                                     s["sink"], s["recent"], query_start_loc=start, ws=s["ws"])
    return pkv.paged_attention_sparse(s["out"], s["q"], s["k_cache"], s["v_cache"], h,
                                      s["block_tables"], s["context_lens"], s["selected"],
                                      query_start_loc=start)


# ----------------------------------------------------------------------------
# what a pass cannot do without (expected values over the lengths' ranges)
# ----------------------------------------------------------------------------
def _mean_blocks(lo, hi):
    return ((lo + hi) / 2 + (BS - 1) / 2) / BS


def work(case):
    n = case["seqs"]
    if case["op"] == "tables":
        width = -(-(case["hi"] + case["chunk"]) // BS)
        tokens = (n - case["chunks"]) + case["chunks"] * case["chunk"]
        new = (n - case["chunks"]) + case["chunks"] * case["chunk"] * 0.75
        held = n * _mean_blocks(case["lo"], case["hi"])
        # table rows, free ids, rows, lengths in; tables, new entries, lengths, slots out
        return dict(bytes=4 * held + 4 * new / BS + 12 * n + 4 * n * width + 4 * new / BS + 8 * n
                    + 12 * tokens + 12, flops=0)
    if case["op"] == "bounds":
        es = 4 if case["dtype"] == "f32" else 2
        new = (case["new_lo"] + case["new_hi"]) / 2
        blocks = n * (new / BS + (BS - 1) / BS)
        rows = n * (new + (BS - 1) / 2)        # a block that was open is read from its start
        kv, d = case["kv_heads"], case["head_dim"]
        return dict(bytes=rows * kv * d * es + blocks * (kv * (2 * d + 1) + 4) + 8 * n,
                    flops=2 * rows * kv * d)
    q, kv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    es = 4 if case["dtype"] == "f32" else 2
    lo, hi = max(case["lo"], case["qlen"]), max(case["hi"], case["qlen"])
    blocks = _mean_blocks(lo, hi)
    rows = n * case["qlen"]
    if case["op"] == "select":
        # the query tokens of one request read the same bounds
        return dict(bytes=n * blocks * (kv * (2 * d + 1) + 4) + rows * (q * d * es
                    + 4 * kv * case["top_k"]) + 4 * n, flops=2 * rows * blocks * q * 2 * d)
    # the shorter contexts of a range have fewer blocks than top_k
    ks = [min(case["top_k"], -(-(lo + (hi - lo) * i // 256) // BS)) for i in range(257)]
    kept = sum(ks) / len(ks)
    # rows of one request have lists of their own: each list's blocks are read
    return dict(bytes=rows * (kv * kept * (2 * BS * d * es + 4) + 2 * q * d * es) + 4 * n,
                flops=4 * rows * q * kept * BS * d)


# ----------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms
# ----------------------------------------------------------------------------
def _exact_tables(s):
    """Request by request, as a pool with a stack of free ids would do it."""
    table = s["table"].cpu().numpy().astype(np.int64)
    stack = s["free_list"].cpu().numpy()[:int(s["free_count"][0])].tolist()
    rows, cached, new = (s[k].cpu().tolist() for k in ("seq_rows", "cached_lens", "new_lens"))
    out = np.full(tuple(s["block_tables"].shape), -1, np.int64)
    slots = np.full(s["slot_mapping"].numel(), -1, np.int64)
    posn = np.zeros(s["slot_mapping"].numel(), np.int64)
    start, ctx = [0], []
    for i, r in enumerate(rows):
        total = cached[i] + new[i]
        for b in range(-(-cached[i] // BS), -(-total // BS)):
            table[r, b] = stack.pop()
        blocks = -(-total // BS)
        out[i, :blocks] = table[r, :blocks]
        p = np.arange(cached[i], total)
        slots[start[-1]:start[-1] + new[i]] = table[r, p // BS] * BS + p % BS
        posn[start[-1]:start[-1] + new[i]] = p
        start.append(start[-1] + new[i])
        ctx.append(total)

    def i32(x):
        return torch.as_tensor(np.asarray(x), dtype=torch.int32)

    return dict(table=i32(table), block_tables=i32(out), context_lens=i32(ctx),
                query_start_loc=i32(start), slot_mapping=torch.from_numpy(slots),
                positions=i32(posn), free_count=i32([len(stack)]))


def _exact_exponent(amax):
    e = np.full(amax.shape, -50.0)
    at = amax > 0
    e[at] = np.ceil(np.log2(amax[at] / 127.0))
    e[at] += amax[at] > 127.0 * 2.0 ** e[at]   # a rounded logarithm, put right
    e[at] -= amax[at] <= 127.0 * 2.0 ** (e[at] - 1)
    return np.clip(e, -50, 50)


def _exact_bounds(s):
    codes, exps = s["bounds"].cpu().numpy().copy(), s["exps"].cpu().numpy().copy()
    tables, ctx = s["block_tables"].cpu().numpy(), s["context_lens"].cpu().tolist()
    start = s["query_start_loc"].cpu().tolist()
    cache = s["k_cache"].cpu()
    for i, c in enumerate(ctx):
        first = (c - (start[i + 1] - start[i])) // BS
        for b in range(first, -(-c // BS)):
            p = int(tables[i, b])
            k = cache[p, :, :min(BS, c - b * BS)].double().numpy()
            hi, lo = k.max(1), k.min(1)
            e = _exact_exponent(np.abs(k).max((1, 2)))
            unit = 2.0 ** e[:, None]
            codes[p, :, 0] = np.clip(np.ceil(hi / unit), -127, 127)
            codes[p, :, 1] = np.clip(np.floor(lo / unit), -127, 127)
            exps[p] = e
    return dict(bounds=torch.from_numpy(codes), exps=torch.from_numpy(exps))


def _exact_select(s):
    """Row by row: sum over d of max(q_d hi_d, q_d lo_d) with the 8-bit values."""
    seq, keys = _row_layout(s)
    kv, d, g = s["kv_heads"], s["head_dim"], s["q_heads"] // s["kv_heads"]
    out = torch.full_like(s["selected"], -1)
    q = s["q"].double().cpu().numpy()
    eq = _exact_exponent(np.abs(q).max(-1))
    code = np.rint(q / 2.0 ** eq[..., None])
    qv = torch.from_numpy(code * 2.0 ** eq[..., None]).to(s["q"].device).view(-1, kv, g, d)
    seq, keys = seq.tolist(), keys.tolist()
    held, last = None, -1
    for r, (i, c) in enumerate(zip(seq, keys)):
        blocks = -(-c // BS)
        if i != last:
            ids = s["block_tables"][i].long().clamp(min=0)
            unit = torch.pow(2.0, s["exps"][ids].double())[:, :, None]
            held, last = (s["bounds"][ids, :, 0].double() * unit,
                          s["bounds"][ids, :, 1].double() * unit), i
        score = torch.full((kv, blocks), -math.inf, dtype=torch.float64, device=s["q"].device)
        for h in range(g):
            qh = qv[r, :, h]
            best = torch.maximum(qh * held[0][:blocks], qh * held[1][:blocks]).sum(-1)
            score = torch.maximum(score, best.t())
        score[:, :s["sink"]] = math.inf
        score[:, max(0, blocks - s["recent"]):] = math.inf
        n = min(blocks, s["top_k"])
        # the n first of (score from above, index from below), then by index
        order = np.lexsort((np.broadcast_to(np.arange(blocks), (kv, blocks)),
                            -score.cpu().numpy()), axis=-1)[:, :n]
        out[r, :, :n] = torch.from_numpy(np.sort(order, -1)).int()
    return out


def _exact_attend(s):
    seq, keys = _row_layout(s)
    kv, d, g = s["kv_heads"], s["head_dim"], s["q_heads"] // s["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    heads = torch.arange(kv, device=s["q"].device)[:, None]
    for r, (i, c) in enumerate(zip(seq.tolist(), keys.tolist())):
        n = min(s["selected"].shape[2], -(-c // BS))     # the list's entries in front of its -1
        ids = s["selected"][r, :, :n].long()
        phys = s["block_tables"][i].long()[ids]
        k = s["k_cache"][phys, heads].double().reshape(kv, n * BS, d)
        v = s["v_cache"][phys, heads].double().reshape(kv, n * BS, d)
        at = (ids[:, :, None] * BS + torch.arange(BS, device=ids.device)).reshape(kv, n * BS)
        x = torch.einsum("hgd,hkd->hgk", s["q"][r].double().view(kv, g, d), k) / math.sqrt(d)
        x = x.masked_fill((at >= c)[:, None], -math.inf)
        out[r] = torch.einsum("hgk,hkd->hgd", torch.softmax(x, -1), v).reshape(-1, d)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "bounds": _exact_bounds, "select": _exact_select,
            "attend": _exact_attend}[case["op"]](s)
