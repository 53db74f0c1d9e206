"""Measured cases of the dense paged cache: the page plan of a step, the store of new keys and values, and
the attention of one new token per sequence over the pages.

``run`` computes each operator in its plain form (elementary torch operations) or, with ``own`` set, through
the library's calls.  Pages hold 16 tokens; a tile is one page of one KV head: 16 key rows, 16 value rows and,
with 8-bit elements, 16 + 16 power-of-two exponents.
"""
import math
import random

import torch

own = False

PAGE = 16
RING = 128
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user, a short chat: the latency of a single decode step (16 query / 4 KV heads)
        dict(name="attend_1x1k_f16", op="attend", batch=1, lo=1024, hi=1024, hq=16, hkv=4, d=128, dtype="f16", bits=16, window=0),
        # a full batch at 32K context with 28 query / 4 KV heads, the shape of the library's main benchmark
        dict(name="attend_8x32k_bf16", op="attend", batch=8, lo=32768, hi=32768, hq=28, hkv=4, d=128, dtype="bf16", bits=16, window=0),
        # long ragged contexts up to 128K, 40 query / 8 KV heads
        dict(name="attend_16xragged_f16", op="attend", batch=16, lo=1024, hi=131072, hq=40, hkv=8, d=128, dtype="f16", bits=16, window=0),
        # the same kind of serving load with an 8-bit cache and bf16 queries
        dict(name="attend_64xragged_e4m3", op="attend", batch=64, lo=500, hi=16001, hq=32, hkv=8, d=128, dtype="bf16", bits=8, window=0),
        # many short requests, one query head per KV head, some rows of the batch empty
        dict(name="attend_256xshort_d64", op="attend", batch=256, lo=0, hi=512, hq=8, hkv=8, d=64, dtype="f16", bits=16, window=0),
        # wide heads at 64K context behind a sliding window
        dict(name="attend_4x64k_d256_window", op="attend", batch=4, lo=65536, hi=65536, hq=8, hkv=8, d=256, dtype="bf16", bits=16, window=4096),
        # the write of one decode step, rows cut out of a fused projection's output
        dict(name="store_64_f16", op="store", tokens=64, pad=0, hkv=8, d=128, dtype="f16", bits=16, blocks=4096),
        # prefill of 32K tokens into a 16-bit cache, the batch's token buffer padded
        dict(name="store_32k_bf16", op="store", tokens=32768, pad=257, hkv=8, d=128, dtype="bf16", bits=16, blocks=4096),
        # the same prefill quantised into an 8-bit cache
        dict(name="store_32k_e4m3", op="store", tokens=32768, pad=257, hkv=8, d=128, dtype="bf16", bits=8, blocks=4096),
        # the plan of one decode step of 64 requests
        dict(name="plan_64_decode", op="plan", batch=64, lo=100, hi=32000, new=1, ended=0, max_tokens=64, max_blocks=2048, ring=0),
        # 1024 requests, mixed prefill chunks and decode tokens, some of them ended; ring of exact recent tokens
        dict(name="plan_1024_mixed", op="plan", batch=1024, lo=0, hi=8000, new=257, ended=31, max_tokens=200000, max_blocks=1024, ring=128),
        # first prefill of 32 prompts of 32K tokens
        dict(name="plan_32x32k_prefill", op="plan", batch=32, lo=0, hi=0, new=32768, ended=0, max_tokens=1048576, max_blocks=2048, ring=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "store", "plan"])
    if op == "attend":
        hkv = rng.choice([1, 2, 3, 4, 8])
        rep = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        d = rng.choice([64, 128, 128, 256, 512])
        batch = _log_int(rng, 1, 200)
        # tokens x heads x d stay below the largest listed case
        most = max(64, min(131072, 400_000_000 // (batch * hkv * d)))
        hi = _log_int(rng, 1, most)
        return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, hq=hkv * rep, hkv=hkv, d=d,
                    dtype=rng.choice(["f16", "bf16"]), bits=rng.choice([16, 16, 8]),
                    window=rng.choice([0, 0, 1 + _log_int(rng, 1, 9000)]))
    if op == "store":
        d, hkv = rng.choice([64, 128, 256, 512]), rng.choice([1, 2, 4, 5, 8])
        tokens = _log_int(rng, 1, 32768 * 128 * 8 // (d * hkv))
        return dict(op=op, tokens=tokens, pad=rng.randint(0, 300), hkv=hkv, d=d, dtype=rng.choice(["f16", "bf16"]),
                    bits=rng.choice([16, 8]), blocks=(tokens + PAGE - 1) // PAGE + rng.randint(0, 900))
    batch = _log_int(rng, 1, 2000)
    new = _log_int(rng, 1, max(2, 1048576 // batch))
    hi = rng.randint(0, 16000)
    return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, new=new, ended=rng.choice([0, 0, 7, 40]),
                max_tokens=batch * new + rng.randint(0, 500), max_blocks=(hi + new + PAGE - 1) // PAGE + rng.randint(0, 40),
                ring=rng.choice([0, 0, 128]))


def _spread(n, lo, hi, shift=0.5):
    """n whole numbers spread evenly over [lo, hi] in a scrambled order (the golden-ratio sequence)."""
    return [lo + int(((i + shift) * 0.6180339887498949) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _lengths(case):
    return _spread(case["batch"], case["lo"], case["hi"])


def _new_lengths(case):
    if case["lo"] == case["hi"] == 0:  # a first prefill: full prompts, the last one odd
        return [case["new"]] * (case["batch"] - 1) + [max(1, case["new"] - 5)]
    new = _spread(case["batch"], 1, case["new"], 0.25)
    if case["ended"]:
        new = [-1 if i % case["ended"] == case["ended"] - 1 else x for i, x in enumerate(new)]
    return new


def _pages(tokens, ring):
    """Pages that hold a sequence of this many tokens; with a ring the newest 1..128 tokens are not in pages."""
    if ring:
        return max(tokens - 1, 0) // RING * (RING // PAGE)
    return (tokens + PAGE - 1) // PAGE


# ---------------------------------------------------------------- inputs
def _two_to(e):
    """2^e in 32 bits for whole e in [-126, 127], without a rounding."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _split_exponent(x):
    """(codes, exponents) of the 8-bit form of x [..., d]: e = the least whole number with max|x| <= 448 * 2^e."""
    m, p = torch.frexp(x.abs().amax(-1).double() / 448.0)
    e = torch.where(m == 0.5, p - 1, p).clamp(-120, 120)  # m in [0.5, 1): max|x| / 448 = m 2^p
    codes = (x.float() * _two_to(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes, e.to(torch.int8)


class _State:
    pass


def _context(case, st):
    """The handle and workspace a user's program keeps."""
    import kv_cache_quantization_tq_gb300 as tq

    if case["op"] == "plan":
        return tq.Context(tq.TQ_LAYOUT_DENSE, 128, 8, 8)
    fmt = tq.TQ_ELEM_BF16 if case["dtype"] == "bf16" else tq.TQ_ELEM_F16
    ctx = tq.Context(tq.TQ_LAYOUT_DENSE, case["d"], case.get("hq", case["hkv"]), case["hkv"], key_bits=case["bits"],
                     value_bits=case["bits"], key_format=fmt)
    if case["op"] == "attend":
        st.workspace = torch.empty(ctx.paged_workspace_size(case["batch"]), dtype=torch.uint8, device="cuda")
    return ctx


def _tile_bytes(case):
    return 2 * PAGE * case["d"] * case["bits"] // 8 + (2 * PAGE if case["bits"] == 8 else 0)


def _fill_pool(case, blocks, gen):
    """A pool of `blocks` pages of keys and values: normal entries, a few strong key channels, and a log-normal
    size of each vector."""
    hkv, d = case["hkv"], case["d"]
    pool = torch.empty(blocks, hkv, _tile_bytes(case), dtype=torch.uint8, device="cuda")
    gain = torch.ones(2, hkv, 1, d, device="cuda")
    gain[:, :, :, torch.randperm(d, generator=gen, device="cuda")[:4]] = 4.0
    part = max(1, (1 << 27) // (hkv * 2 * PAGE * d))
    for i in range(0, blocks, part):
        n = min(part, blocks - i)
        x = torch.randn(n, hkv, 2, PAGE, d, generator=gen, device="cuda")
        x *= gain.permute(1, 0, 2, 3)
        x *= torch.exp(0.5 * torch.randn(n, hkv, 2, PAGE, 1, generator=gen, device="cuda"))
        if case["bits"] == 16:
            pool[i:i + n] = x.to(DTYPES[case["dtype"]]).view(torch.uint8).reshape(n, hkv, -1)
        else:
            codes, e = _split_exponent(x)
            pool[i:i + n, :, :2 * PAGE * d] = codes.view(torch.uint8).reshape(n, hkv, -1)
            pool[i:i + n, :, 2 * PAGE * d:] = e.view(torch.uint8).reshape(n, hkv, -1)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 13)
    st = _State()
    st.case = case
    i32 = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "attend":
        lens = _lengths(case)
        st.max_blocks = max(1, (max(lens) + PAGE - 1) // PAGE)
        used = [(n + PAGE - 1) // PAGE for n in lens]
        blocks = sum(used) + 3
        st.pool = _fill_pool(case, blocks, gen)
        ids = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
        first = torch.tensor([sum(used[:b]) for b in range(len(used))], device="cuda")
        held = torch.tensor(used, device="cuda")
        j = torch.arange(st.max_blocks, device="cuda")[None, :]
        at = (first[:, None] + j).clamp(max=blocks - 1)
        st.block_table = torch.where(j < held[:, None], ids[at], torch.full((), -1, **i32)).contiguous()
        st.lengths = torch.tensor(lens, **i32)
        # what lies behind a sequence's last token is whatever the memory held: here the bit pattern of a NaN
        for b, n in enumerate(lens[:32]):
            if n % PAGE:
                tile = st.pool[int(st.block_table[b, n // PAGE])]
                rows = tile[:, :_tile_bytes(case) // (2 * PAGE) * 2 * PAGE][:, :2 * PAGE * case["d"] * case["bits"] // 8]
                rows.view(case["hkv"], 2, PAGE, -1)[:, :, n % PAGE:] = 0xFF
        st.q = torch.randn(case["batch"], case["hq"], case["d"], generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        st.out = torch.empty(case["batch"], case["hq"], case["d"], dtype=torch.float32, device="cuda")
        st.lse = torch.empty(case["batch"], case["hq"], dtype=torch.float32, device="cuda")
    elif case["op"] == "store":
        n, hkv, d = case["tokens"], case["hkv"], case["d"]
        # keys and values are columns of one projection's output [tokens, q | k | v]
        wide = torch.randn(n + case["pad"], (2 * hkv + hkv) * d, generator=gen, device="cuda")
        wide *= torch.exp(0.5 * torch.randn(n + case["pad"], 1, generator=gen, device="cuda"))
        st.wide = wide.to(DTYPES[case["dtype"]])
        st.k = st.wide[:, hkv * d:2 * hkv * d].view(-1, hkv, d)
        st.v = st.wide[:, 2 * hkv * d:].view(-1, hkv, d)
        st.pool = _fill_pool(case, case["blocks"], gen)
        # whole pages in a random order, as a plan gives them; padded rows have no slot
        page = torch.randperm(case["blocks"], generator=gen, device="cuda")[:(n + PAGE - 1) // PAGE]
        t = torch.arange(n, device="cuda")
        st.slots = torch.full((n + case["pad"],), -1, dtype=torch.int64, device="cuda")
        st.slots[:n] = page[t // PAGE] * PAGE + t % PAGE
    else:
        ctx_len, new, ring = _lengths(case), _new_lengths(case), case["ring"]
        if any(n < 0 for n in new):
            ctx_len = [max(c, 1) if n < 0 else c for c, n in zip(ctx_len, new)]
        held = [_pages(c, ring) for c in ctx_len]
        need = sum(_pages(c + max(n, 0), ring) - h for c, n, h in zip(ctx_len, new, held))
        st.blocks = sum(held) + need + 64
        ids = torch.randperm(st.blocks, generator=gen, device="cuda").to(torch.int32)
        st.block_table = torch.full((case["batch"], case["max_blocks"]), -1, **i32)
        first = torch.tensor([sum(held[:b]) for b in range(len(held))], device="cuda")
        h = torch.tensor(held, device="cuda")
        j = torch.arange(case["max_blocks"], device="cuda")[None, :]
        at = (first[:, None] + j).clamp(max=st.blocks - 1)
        st.block_table = torch.where(j < h[:, None], ids[at], st.block_table).contiguous()
        # the free pages stand in a circular queue, from a head that earlier steps have moved on
        st.queue = torch.full((st.blocks,), -1, **i32)
        free = ids[sum(held):]
        head = int(seed) * 131 % st.blocks
        st.queue[(head + torch.arange(free.numel(), device="cuda")) % st.blocks] = free
        st.queue_state = torch.tensor([head, free.numel()], **i32)
        st.ctx_len, st.new_len = torch.tensor(ctx_len, **i32), torch.tensor(new, **i32)
        st.lengths = torch.empty(case["batch"], **i32)
        st.n_paged, st.n_ring = torch.empty(case["batch"], **i32), torch.empty(case["batch"], **i32)
        st.token_start = torch.empty(case["batch"] + 1, **i32)
        st.slots = torch.empty(case["max_tokens"], dtype=torch.int64, device="cuda")
        st.positions, st.rows = torch.empty(case["max_tokens"], **i32), torch.empty(case["max_tokens"], **i32)
        st.queue_state_out = torch.empty(2, **i32)
    if own:
        st.ctx = _context(case, st)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    return {"attend": _run_attend, "store": _run_store, "plan": _run_plan}[st.case["op"]](st)


def _run_attend(st):
    case = st.case
    if own:
        st.ctx.paged_attention(st.q, st.pool, st.block_table, st.lengths, st.out, st.workspace, lse=st.lse, window=case["window"])
        return {"out": st.out, "lse": st.lse}
    bsz, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    tiles = st.pool[st.block_table.long().clamp(min=0)]  # [batch, pages, hkv, tile]
    k, v = _rows(case, tiles)                             # [batch, hkv, tokens, d] in 32 bits
    pos = torch.arange(k.shape[2], device="cuda")[None, :]
    n = st.lengths.long()[:, None]
    seen = (pos < n) & (pos >= (n - case["window"] if case["window"] else 0))
    v = torch.where(seen[:, None, :, None], v, 0.0)
    q = st.q.float().view(bsz, hkv, hq // hkv, d)
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    s = torch.where(seen[:, None, None, :], s, -torch.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return {"out": out.view(bsz, hq, d), "lse": (top + torch.log(total)).view(bsz, hq)}


def _rows(case, tiles):
    """Keys and values [batch, hkv, tokens, d] in 32 bits of tiles [batch, pages, hkv, bytes]."""
    bsz, pages, hkv, d = tiles.shape[0], tiles.shape[1], tiles.shape[2], case["d"]
    if case["bits"] == 16:
        x = tiles.view(DTYPES[case["dtype"]]).view(bsz, pages, hkv, 2, PAGE, d)
        x = x.permute(3, 0, 2, 1, 4, 5).float()
    else:
        c = tiles[..., :2 * PAGE * d].contiguous().view(torch.float8_e4m3fn).view(bsz, pages, hkv, 2, PAGE, d).float()
        e = tiles[..., 2 * PAGE * d:].contiguous().view(torch.int8).view(bsz, pages, hkv, 2, PAGE, 1)
        x = (c * _two_to(e)).permute(3, 0, 2, 1, 4, 5)
    x = x.reshape(2, bsz, hkv, pages * PAGE, d)
    return x[0], x[1]


def _pool_views(case, pool):
    """The pool's contents as the numbers they are."""
    nb, hkv, d = pool.shape[0], case["hkv"], case["d"]
    if case["bits"] == 16:
        return {"rows": pool.view(DTYPES[case["dtype"]]).view(nb, hkv, 2, PAGE, d)}
    return {"codes": pool[..., :2 * PAGE * d].view(torch.float8_e4m3fn), "exponents": pool[..., 2 * PAGE * d:].view(torch.int8)}


def _run_store(st):
    case = st.case
    if own:
        st.ctx.paged_store(st.k, st.v, st.slots, st.pool)
        return _pool_views(case, st.pool)
    d = case["d"]
    at = st.slots >= 0
    block, t = st.slots[at] // PAGE, st.slots[at] % PAGE
    x = torch.stack([st.k[at], st.v[at]], 2)  # [tokens, hkv, 2, d]
    if case["bits"] == 16:
        rows = st.pool.view(x.dtype).view(-1, case["hkv"], 2, PAGE, d)
        rows[block, :, :, t] = x
    else:
        codes, e = _split_exponent(x.float())
        st.pool[..., :2 * PAGE * d].unflatten(-1, (2, PAGE, d))[block, :, :, t] = codes.view(torch.uint8)
        st.pool[..., 2 * PAGE * d:].unflatten(-1, (2, PAGE))[block, :, :, t] = e.view(torch.uint8)
    return _pool_views(case, st.pool)


def _held(tokens, ring):
    return (tokens - 1).clamp(min=0) // RING * (RING // PAGE) if ring else (tokens + PAGE - 1) // PAGE


def _run_plan(st):
    case = st.case
    out = dict(block_table=st.block_table, lengths=st.lengths, n_paged=st.n_paged, n_ring=st.n_ring, token_start=st.token_start,
               slots=st.slots, positions=st.positions, rows=st.rows, queue=st.queue, queue_state=st.queue_state_out)
    if own:
        st.ctx.plan_pages(st.ctx_len, st.new_len, st.block_table, st.queue, st.queue_state, st.lengths, st.token_start, st.slots,
                          st.queue_state_out, num_blocks=st.blocks, positions=st.positions, rows=st.rows, n_paged=st.n_paged,
                          n_ring=st.n_ring, ring_capacity=case["ring"])
        return out
    ring, cap, bsz, maxb = case["ring"], st.queue.numel(), case["batch"], case["max_blocks"]
    ctx, new = st.ctx_len.long(), st.new_len.long()
    head, count = st.queue_state.long()
    add, ended = new.clamp(min=0), new < 0
    old, total = _held(ctx, ring), ctx + add
    need = torch.where(ended, 0, _held(total, ring) - old)
    token_end, page_end = add.cumsum(0), need.cumsum(0)
    token_start, page_start = token_end - add, page_end - need
    fits = (token_end <= case["max_tokens"]) & ((need == 0) | (page_end <= count)) & (_held(total, ring) <= maxb)
    length = torch.where(ended, 0, torch.where(fits, total, ctx))
    taken = torch.where(fits, need, 0).sum()
    # new pages: entry j of a row, old[b] <= j < old[b] + need[b], is the queue's entry page_start[b] + j - old[b]
    j = torch.arange(maxb, device="cuda")[None, :]
    grown = fits[:, None] & (j >= old[:, None]) & (j < (old + need)[:, None])
    k = (head + page_start[:, None] + j - old[:, None]) % cap
    st.block_table.copy_(torch.where(grown, st.queue[k], st.block_table))
    # one entry per new token, in the order of the requests
    i = torch.arange(case["max_tokens"], device="cuda")
    b = torch.searchsorted(token_end, i, right=True).clamp(max=bsz - 1)
    real = i < token_end[-1]
    pos = ctx[b] + i - token_start[b]
    paged = torch.where(ended, 0, (length - 1).clamp(min=0) // RING * RING if ring else length)
    into = real & fits[b] & (pos < paged[b])
    block = st.block_table[b, (pos // PAGE).clamp(max=maxb - 1)].long()
    st.slots.copy_(torch.where(into, block * PAGE + pos % PAGE, -1))
    st.positions.copy_(torch.where(real, pos, -1))
    st.rows.copy_(torch.where(real, b, -1))
    # the pages of ended requests go to the queue's end
    back = torch.where(ended, old, 0)
    back_start = back.cumsum(0) - back
    r = torch.where(ended[:, None] & (j < old[:, None]), (head + count + back_start[:, None] + j) % cap, cap)
    wide = torch.cat([st.queue, st.queue[:1]])
    wide[r.flatten()] = st.block_table.flatten()
    st.queue.copy_(wide[:cap])
    st.lengths.copy_(length)
    st.n_paged.copy_(paged)
    st.n_ring.copy_(length - paged)
    st.token_start.copy_(torch.cat([token_start, token_end[-1:]]))
    st.queue_state_out.copy_(torch.stack([(head + taken) % cap, count - taken + back.sum()]))
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "attend":
        lens = [min(n, case["window"]) if case["window"] else n for n in _lengths(case)]
        per = 2 * case["d"] * case["bits"] // 8 + (2 if case["bits"] == 8 else 0)
        rows = case["batch"] * case["hq"]
        cache = sum(lens) * case["hkv"] * per + sum((n + PAGE - 1) // PAGE for n in lens) * 4
        return {"bytes": cache + rows * (case["d"] * 6 + 4) + 4 * case["batch"], "flops": 4.0 * sum(lens) * case["hq"] * case["d"]}
    if case["op"] == "store":
        vectors = 2 * case["tokens"] * case["hkv"]
        written = case["d"] * case["bits"] // 8 + (1 if case["bits"] == 8 else 0)
        return {"bytes": vectors * (2 * case["d"] + written) + 8 * (case["tokens"] + case["pad"]), "flops": 0}
    ctx, new, ring = _lengths(case), _new_lengths(case), case["ring"]
    grown = sum(_pages(c + n, ring) - _pages(c, ring) for c, n in zip(ctx, new) if n > 0)
    back = sum(_pages(c, ring) for c, n in zip(ctx, new) if n < 0)
    return {"bytes": 16 * case["max_tokens"] + 8 * (grown + back) + 24 * case["batch"] + 16, "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    st = prepare(case, seed)
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "store":
        return _exact_store(case, st)
    rep = case["hq"] // hkv
    out = torch.zeros(case["batch"], case["hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], case["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n <= lo:
            continue
        p = torch.arange(lo, n, device="cuda")
        block, t = st.block_table[b].long()[p // PAGE], p % PAGE
        for h in range(hkv):
            tile = st.pool[:, h]
            if case["bits"] == 16:
                x = tile.view(DTYPES[case["dtype"]]).view(-1, 2, PAGE, d)
                k, v = x[block, 0, t].double(), x[block, 1, t].double()
            else:
                c = tile[:, :2 * PAGE * d].unflatten(1, (2, PAGE, d))
                e = tile[:, 2 * PAGE * d:].view(torch.int8).unflatten(1, (2, PAGE))
                k, v = (c[block, i, t].view(torch.float8_e4m3fn).double() * _power(e[block, i, t])[:, None] for i in (0, 1))
            for g in range(h * rep, (h + 1) * rep):
                s = (k * st.q[b, g].double()).sum(1) / math.sqrt(d)
                lse[b, g] = torch.logsumexp(s, 0)
                out[b, g] = (torch.exp(s - lse[b, g])[:, None] * v).sum(0)
    return {"out": out, "lse": lse}


def _power(e):
    """2^e in 64 bits for whole e, without a rounding."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_store(case, st):
    d = case["d"]
    if case["bits"] == 16:
        rows = _pool_views(case, st.pool)["rows"].double()
    else:
        rows = st.pool[..., :2 * PAGE * d].view(torch.float8_e4m3fn).double().unflatten(-1, (2, PAGE, d))
    for i, x in enumerate((st.k, st.v)):
        x = x[:case["tokens"]].double()
        if case["bits"] == 8:
            # scaled so that the largest entry is at most 448, then rounded to 3 fraction bits (ties to even), at
            # least a multiple of 2^-9
            top = x.abs().amax(2, keepdim=True)
            e = torch.full_like(top, -120, dtype=torch.int64)
            for k in range(-120, 120):  # the least e with top <= 448 * 2^e
                e = torch.where(top > 448.0 * 2.0 ** k, k + 1, e)
            x = x / _power(e)
            step = torch.full_like(x, 2.0 ** -9)
            for k in range(-6, 9):
                step = torch.where(x.abs() >= 2.0 ** k, 2.0 ** (k - 3), step)
            x = torch.round(x / step) * step
        slot = st.slots[:case["tokens"]]
        rows[slot // PAGE, :, i, slot % PAGE] = x
    return {"rows": rows} if case["bits"] == 16 else {"codes": rows.flatten(2), "exponents": None}
