"""Measured cases of the small cache: 4-bit pages (store and single-token attention), attention whose scores are
capped and biased by distance, the accumulation of attention weights per cached token, and the eviction of the
tokens that had least of it.

``run`` computes each operator in its plain form (elementary torch operations) or, with ``own`` set, through
the library's calls.  Pages hold 16 tokens; a tile is one page of one KV head: 16 key rows, 16 value rows, then
with 4-bit elements the block scales of the keys and of the values, and with 4- and 8-bit elements 16 + 16
power-of-two exponents.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
BLOCK = 16  # 4-bit elements that share a scale
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user, a short chat from a 4-bit cache: the latency of a single decode step (16 query / 4 KV heads)
        dict(name="attend4_1x1k", op="attend", batch=1, lo=1024, hi=1024, hq=16, hkv=4, d=128, dtype="f16", bits=4, window=0, cap=0.0, slopes=False),
        # a serving load of ragged contexts up to 16K, 32 query / 8 KV heads, from a 4-bit cache
        dict(name="attend4_64xragged", op="attend", batch=64, lo=500, hi=16001, hq=32, hkv=8, d=128, dtype="bf16", bits=4, window=0, cap=0.0, slopes=False),
        # a full batch at 32K context with wide heads from a 4-bit cache
        dict(name="attend4_8x32k_d256", op="attend", batch=8, lo=32768, hi=32768, hq=40, hkv=8, d=256, dtype="f16", bits=4, window=0, cap=0.0, slopes=False),
        # one user, scores biased by distance, one query head per KV head
        dict(name="scored_1x2k_slopes", op="attend", batch=1, lo=2048, hi=2048, hq=8, hkv=8, d=64, dtype="f16", bits=16, window=0, cap=0.0, slopes=True),
        # a full batch at 32K context (28 query / 4 KV heads), capped scores
        dict(name="scored_8x32k_cap", op="attend", batch=8, lo=32768, hi=32768, hq=28, hkv=4, d=128, dtype="bf16", bits=16, window=0, cap=50.0, slopes=False),
        # ragged contexts from an 8-bit cache, scores capped and biased by distance
        dict(name="scored_64xragged_both_e4m3", op="attend", batch=64, lo=500, hi=16001, hq=32, hkv=8, d=128, dtype="bf16", bits=8, window=0, cap=30.0, slopes=True),
        # the write of one decode step into a 4-bit cache, rows cut out of a fused projection's output
        dict(name="store4_64", op="store", tokens=64, pad=0, hkv=8, d=128, dtype="f16", bits=4, blocks=512),
        # prefill of 32K tokens into a 4-bit cache, the batch's token buffer padded
        dict(name="store4_32k", op="store", tokens=32768, pad=257, hkv=8, d=128, dtype="bf16", bits=4, blocks=2048),
        # the weights of one decode step of one user added up per cached token
        dict(name="weights_1x4k", op="weights", batch=1, lo=4096, hi=4096, hq=16, hkv=4, d=128, dtype="f16", bits=16, window=0, cap=0.0, slopes=False, decay=1.0),
        # the same for a serving load of ragged contexts from a 4-bit cache, older weights fading
        dict(name="weights_64xragged_4bit", op="weights", batch=64, lo=500, hi=16001, hq=32, hkv=8, d=128, dtype="bf16", bits=4, window=0, cap=0.0, slopes=False, decay=0.875),
        # a prompt of 32K tokens cut down to 2K before the answer begins
        dict(name="evict_1x32k_to_2k", op="evict", batch=1, lo=32768, hi=32768, keep=2048, sinks=4, recent=256, hkv=8, d=128, dtype="f16", bits=16),
        # a full batch held at 4K tokens: every sequence gives up to 256 back, from an 8-bit cache
        dict(name="evict_64x4k_e4m3", op="evict", batch=64, lo=4097, hi=4352, keep=4096, sinks=4, recent=128, hkv=8, d=128, dtype="bf16", bits=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend4", "scored", "weights", "store", "evict"])
    dtype = rng.choice(["f16", "bf16"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128, 128, 256, 512])
    if op == "store":
        tokens = _log_int(rng, 1, 32768 * 128 * 8 // (d * hkv))
        return dict(op=op, tokens=tokens, pad=rng.randint(0, 300), hkv=hkv, d=d, dtype=dtype, bits=4,
                    blocks=(tokens + PAGE - 1) // PAGE + rng.randint(0, 300))
    if op == "evict":
        batch = _log_int(rng, 1, 64)
        most = max(64, min(65536, 16_000_000 // (batch * hkv * max(1, d // 64))))
        hi = _log_int(rng, 16, most)
        keep = _log_int(rng, 1, min(hi, 8192))
        recent = rng.choice([0, 1, keep // 8, keep // 2])
        return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, keep=keep, sinks=rng.choice([0, 0, 1, 4]), recent=recent,
                    hkv=hkv, d=d, dtype=dtype, bits=rng.choice([16, 8, 4]))
    rep = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    batch = _log_int(rng, 1, 128)
    # tokens x heads x d stay below the largest listed case
    most = max(64, min(65536, 200_000_000 // (batch * hkv * d)))
    hi = _log_int(rng, 1, most)
    case = dict(op="attend", batch=batch, lo=rng.randint(0, hi), hi=hi, hq=hkv * rep, hkv=hkv, d=d, dtype=dtype, bits=4,
                window=rng.choice([0, 0, 1 + _log_int(rng, 1, 9000)]), cap=0.0, slopes=False)
    if op != "attend4":
        kind = rng.choice(["cap", "slopes", "both"]) if op == "scored" else rng.choice(["none", "none", "cap", "slopes", "both"])
        case.update(bits=rng.choice([16, 16, 8, 4]), cap=rng.choice([8.0, 30.0, 50.0]) if kind in ("cap", "both") else 0.0,
                    slopes=kind in ("slopes", "both"))
    if op == "weights":
        case.update(op="weights", decay=rng.choice([1.0, 1.0, 0.875, 0.99]))
    return case


def _spread(n, lo, hi, shift=0.5):
    """n whole numbers spread evenly over [lo, hi] in a scrambled order (the golden-ratio sequence)."""
    return [lo + int(((i + shift) * 0.6180339887498949) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _lengths(case):
    return _spread(case["batch"], case["lo"], case["hi"])


# ---------------------------------------------------------------- number formats
def _two_to(e):
    """2^e in 32 bits for whole e in [-126, 127], without a rounding."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _least_exponent(top, most):
    """The least whole number e in [-120, 120] with top <= most * 2^e."""
    m, p = torch.frexp(top.double() / most)
    return torch.where(m == 0.5, p - 1, p).clamp(-120, 120)  # m in [0.5, 1): top / most = m 2^p


def _split8(x):
    """(codes, exponents) of the 8-bit form of x [..., d]: e = the least whole number with max|x| <= 448 * 2^e."""
    e = _least_exponent(x.abs().amax(-1), 448.0)
    codes = (x.float() * _two_to(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes, e.to(torch.int8)


def _split4(x):
    """(codes, scales, exponents) of the 4-bit form of x [..., d]: e = the least whole number with max|x| <= 2688 * 2^e; of
    every 16 elements the scale s = e4m3(max|x| 2^-e / 6) and the codes e2m1(x 2^-e / s), two to a byte."""
    e = _least_exponent(x.abs().amax(-1), 2688.0)
    y = (x.float() * _two_to(-e)[..., None]).unflatten(-1, (-1, BLOCK))
    scales = (y.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    s = scales.float()[..., None]
    y = torch.where(s > 0, y / torch.where(s > 0, s, 1.0), torch.copysign(torch.zeros_like(y), y))
    # magnitudes 0 .5 1 1.5 2 3 4 6: the steps' middles, ties to the even code
    a = y.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = (c + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    return c[..., 0::2] + 16 * c[..., 1::2], scales, e.to(torch.int8)


def _pairs():
    """The two values that a byte of 4-bit codes stands for, for all 256 bytes."""
    m = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    v = torch.cat([m, -m])
    b = torch.arange(256, device="cuda")
    return torch.stack([v[b % 16], v[b // 16]], 1)


def _tile_bytes(bits, d):
    return 64 * d if bits == 16 else 32 * d + 32 if bits == 8 else 18 * d + 32


def _rows(case, tiles, pairs):
    """Keys and values [batch, hkv, tokens, d] in 32 bits of tiles [batch, pages, hkv, bytes]."""
    bsz, pages, hkv, d = tiles.shape[0], tiles.shape[1], tiles.shape[2], case["d"]
    if case["bits"] == 16:
        x = tiles.view(DTYPES[case["dtype"]]).view(bsz, pages, hkv, 2, PAGE, d).permute(3, 0, 2, 1, 4, 5).float()
    elif case["bits"] == 8:
        c = tiles[..., :32 * d].contiguous().view(torch.float8_e4m3fn).view(bsz, pages, hkv, 2, PAGE, d).float()
        e = tiles[..., 32 * d:].contiguous().view(torch.int8).view(bsz, pages, hkv, 2, PAGE, 1)
        x = (c * _two_to(e)).permute(3, 0, 2, 1, 4, 5)
    else:
        c = pairs.index_select(0, tiles[..., :16 * d].flatten().int()).view(bsz, pages, hkv, 2, PAGE, d // BLOCK, BLOCK)
        s = tiles[..., 16 * d:18 * d].contiguous().view(torch.float8_e4m3fn).view(bsz, pages, hkv, 2, PAGE, d // BLOCK, 1).float()
        e = tiles[..., 18 * d:].contiguous().view(torch.int8).view(bsz, pages, hkv, 2, PAGE, 1, 1)
        x = (c * (s * _two_to(e))).flatten(-2).permute(3, 0, 2, 1, 4, 5)
    x = x.reshape(2, bsz, hkv, pages * PAGE, d)
    return x[0], x[1]


def _pool_views(case, pool):
    """The pool's contents as the numbers they are; bytes of 4-bit codes as bytes, which leaves no room for a difference."""
    bits, d = case["bits"], case["d"]
    if bits == 16:
        return {"rows": pool.view(DTYPES[case["dtype"]])}
    if bits == 8:
        return {"codes": pool[..., :32 * d].view(torch.float8_e4m3fn), "exponents": pool[..., 32 * d:].view(torch.int8)}
    return {"codes": pool[..., :16 * d], "scales": pool[..., 16 * d:18 * d].view(torch.float8_e4m3fn), "exponents": pool[..., 18 * d:].view(torch.int8)}


# ---------------------------------------------------------------- inputs
class _State:
    pass


def _context(case, st):
    """The handle and workspace a user's program keeps."""
    import kv_cache_quantization_tq_gb300 as tq

    fmt = tq.TQ_ELEM_BF16 if case["dtype"] == "bf16" else tq.TQ_ELEM_F16
    ctx = tq.Context(tq.TQ_LAYOUT_DENSE, case["d"], case.get("hq", case["hkv"]), case["hkv"], key_bits=case["bits"],
                     value_bits=case["bits"], key_format=fmt)
    if case["op"] == "attend":
        st.workspace = torch.empty(ctx.paged_workspace_size(case["batch"]), dtype=torch.uint8, device="cuda")
    return ctx


def _fill_pool(case, blocks, gen):
    """A pool of `blocks` pages of keys and values: normal entries, a few strong key channels, and a log-normal
    size of each vector."""
    hkv, d, bits = case["hkv"], case["d"], case["bits"]
    pool = torch.empty(blocks, hkv, _tile_bytes(bits, d), dtype=torch.uint8, device="cuda")
    gain = torch.ones(2, hkv, 1, d, device="cuda")
    gain[:, :, :, torch.randperm(d, generator=gen, device="cuda")[:4]] = 4.0
    part = max(1, (1 << 27) // (hkv * 2 * PAGE * d))
    for i in range(0, blocks, part):
        n = min(part, blocks - i)
        x = torch.randn(n, hkv, 2, PAGE, d, generator=gen, device="cuda")
        x *= gain.permute(1, 0, 2, 3)
        x *= torch.exp(0.5 * torch.randn(n, hkv, 2, PAGE, 1, generator=gen, device="cuda"))
        if bits == 16:
            pool[i:i + n] = x.to(DTYPES[case["dtype"]]).view(torch.uint8).reshape(n, hkv, -1)
        elif bits == 8:
            codes, e = _split8(x)
            pool[i:i + n, :, :32 * d] = codes.view(torch.uint8).reshape(n, hkv, -1)
            pool[i:i + n, :, 32 * d:] = e.view(torch.uint8).reshape(n, hkv, -1)
        else:
            codes, s, e = _split4(x)
            pool[i:i + n, :, :16 * d] = codes.reshape(n, hkv, -1)
            pool[i:i + n, :, 16 * d:18 * d] = s.view(torch.uint8).reshape(n, hkv, -1)
            pool[i:i + n, :, 18 * d:] = e.view(torch.uint8).reshape(n, hkv, -1)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 29)
    st = _State()
    st.case = case
    f32, i32 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    hkv, d = case["hkv"], case["d"]
    st.pairs = _pairs() if case["bits"] == 4 else None
    if case["op"] == "store":
        n = case["tokens"]
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
        lens, bsz = _lengths(case), case["batch"]
        st.max_blocks = max(1, (max(lens) + PAGE - 1) // PAGE)
        used = [(n + PAGE - 1) // PAGE for n in lens]
        st.blocks = sum(used) + 3
        st.pool = _fill_pool(case, st.blocks, gen)
        ids = torch.randperm(st.blocks, generator=gen, device="cuda").to(torch.int32)
        first = torch.tensor([sum(used[:b]) for b in range(bsz)], device="cuda")
        held = torch.tensor(used, device="cuda")
        j = torch.arange(st.max_blocks, device="cuda")[None, :]
        at = (first[:, None] + j).clamp(max=st.blocks - 1)
        st.block_table = torch.where(j < held[:, None], ids[at], torch.full((), -1, **i32)).contiguous()
        st.lengths = torch.tensor(lens, **i32)
        n = st.max_blocks * PAGE
        if case["op"] == "evict":
            # sums of weights: a few tokens have most of them, some have none at all, and equal sums occur
            w = torch.exp(2.0 * torch.randn(bsz, hkv, n, generator=gen, device="cuda") - 3.0)
            u = torch.rand(bsz, hkv, n, generator=gen, device="cuda")
            st.weights = torch.where(u < 0.1, 0.0, torch.where(u < 0.3, torch.round(w * 16) / 16, w)).contiguous()
            st.keep = torch.full((bsz,), case["keep"], **i32)
            st.weights_out = torch.zeros(bsz, hkv, n, **f32)
            st.kept = torch.full((bsz, hkv, n), -1, **i32)
            st.lengths_out = torch.zeros(bsz, **i32)
            # the queue of free pages, from a head that earlier steps have moved on
            st.queue = torch.full((st.blocks,), -1, **i32)
            st.queue_state = torch.tensor([int(seed) * 131 % st.blocks, 3], **i32)
            st.queue[(int(seed) * 131 + torch.arange(3, device="cuda")) % st.blocks] = ids[sum(used):]
            st.queue_state_out = torch.zeros(2, **i32)
        else:
            # what lies behind a sequence's last token is whatever the memory held: here the bit pattern of a NaN
            for b, m in enumerate(lens[:32]):
                if m % PAGE:
                    row = case["bits"] * d // 8
                    tile = st.pool[int(st.block_table[b, m // PAGE])]
                    tile[:, :2 * PAGE * row].unflatten(1, (2, PAGE, row))[:, :, m % PAGE:] = 0xFF
                    if case["bits"] == 4:
                        tile[:, 16 * d:18 * d].unflatten(1, (2, PAGE, d // BLOCK))[:, :, m % PAGE:] = 0xFF
            st.q = torch.randn(bsz, case["hq"], d, generator=gen, device="cuda").to(DTYPES[case["dtype"]])
            # slopes 2^(-8 i / heads), the geometric sequence of attention with a linear bias
            i = torch.arange(1, case["hq"] + 1, **f32)
            st.slopes = torch.exp2(-8.0 * i / case["hq"]) if case["slopes"] else None
            if case["op"] == "attend":
                st.out = torch.empty(bsz, case["hq"], d, **f32)
                st.lse = torch.empty(bsz, case["hq"], **f32)
            else:
                st.lse = _log_sum(_scores(st, _keys(st)))  # as the attention of the step leaves it
                st.weights = torch.exp(torch.randn(bsz, hkv, n, generator=gen, device="cuda") - 6.0)
                st.weights_out = torch.zeros(bsz, hkv, n, **f32)
    if own:
        st.ctx = _context(case, st)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    return {"attend": _run_attend, "store": _run_store, "weights": _run_weights, "evict": _run_evict}[st.case["op"]](st)


def _both(st):
    return _rows(st.case, st.pool[st.block_table.long().clamp(min=0)], st.pairs)


def _keys(st):
    return _both(st)[0]


def _seen(st, tokens):
    """[batch, tokens]: the positions that count."""
    pos, n = torch.arange(tokens, device="cuda")[None, :], st.lengths.long()[:, None]
    return (pos < n) & (pos >= (n - st.case["window"] if st.case["window"] else 0))


def _scores(st, k):
    """[batch, hkv, rep, tokens] in 32 bits, -inf where a position does not count."""
    case = st.case
    bsz, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    s = torch.matmul(st.q.float().view(bsz, hkv, hq // hkv, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    if case["slopes"]:
        back = (torch.arange(k.shape[2], device="cuda")[None, :] - (st.lengths.long()[:, None] - 1)).float()
        s = s + st.slopes.view(1, hkv, hq // hkv, 1) * back[:, None, None, :]
    return torch.where(_seen(st, k.shape[2])[:, None, None, :], s, -torch.inf)


def _log_sum(s):
    """ln sum exp over the last axis, [batch, heads]."""
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    return (top + torch.log(torch.exp(s - top).sum(-1, keepdim=True))).reshape(s.shape[0], -1)


def _run_attend(st):
    case = st.case
    if own:
        st.ctx.paged_attention(st.q, st.pool, st.block_table, st.lengths, st.out, st.workspace, lse=st.lse, window=case["window"],
                               cap=case["cap"], slopes=st.slopes)
        return {"out": st.out, "lse": st.lse}
    k, v = _both(st)
    s = _scores(st, k)
    v = torch.where(_seen(st, k.shape[2])[:, None, :, None], v, 0.0)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return {"out": out.view(case["batch"], case["hq"], case["d"]), "lse": (top + torch.log(total)).view(case["batch"], case["hq"])}


def _run_store(st):
    case = st.case
    if own:
        st.ctx.paged_store(st.k, st.v, st.slots, st.pool)
        return _pool_views(case, st.pool)
    d = case["d"]
    at = st.slots >= 0
    block, t = st.slots[at] // PAGE, st.slots[at] % PAGE
    codes, s, e = _split4(torch.stack([st.k[at], st.v[at]], 2))  # [tokens, hkv, 2, ...]
    st.pool[..., :16 * d].unflatten(-1, (2, PAGE, d // 2))[block, :, :, t] = codes
    st.pool[..., 16 * d:18 * d].unflatten(-1, (2, PAGE, d // BLOCK))[block, :, :, t] = s.view(torch.uint8)
    st.pool[..., 18 * d:].unflatten(-1, (2, PAGE))[block, :, :, t] = e.view(torch.uint8)
    return _pool_views(case, st.pool)


def _run_weights(st):
    case = st.case
    if own:
        st.ctx.paged_weights(st.q, st.pool, st.block_table, st.lengths, st.lse, st.weights_out, weights=st.weights, decay=case["decay"],
                             window=case["window"], cap=case["cap"], slopes=st.slopes)
        return st.weights_out
    s = _scores(st, _keys(st))
    p = torch.exp(s - st.lse.view(case["batch"], case["hkv"], -1, 1)).sum(2)
    held = torch.arange(p.shape[2], device="cuda")[None, :] < st.lengths[:, None]
    p = torch.where(_seen(st, p.shape[2])[:, None, :], p, 0.0)
    st.weights_out.copy_(torch.where(held[:, None, :], case["decay"] * st.weights + p, st.weights_out))
    return st.weights_out


def _parts(case):
    """(first byte, bytes of a token) of each part of a tile that holds 16 tokens one behind another."""
    bits, d = case["bits"], case["d"]
    row = bits * d // 8
    parts = [(0, row), (PAGE * row, row)]
    if bits == 4:
        parts += [(16 * d, d // BLOCK), (17 * d, d // BLOCK)]
    if bits < 16:
        end = _tile_bytes(bits, d)
        parts += [(end - 2 * PAGE, 1), (end - PAGE, 1)]
    return parts


def _move(pool, first, size, sb, ss, db, ds, head):
    """Bytes of the tokens at (block, slot) sb, ss go to db, ds."""
    part = pool[..., first:first + PAGE * size].unflatten(-1, (PAGE, size))
    part[db, head, ds] = part[sb, head, ss]


def _run_evict(st):
    case = st.case
    if own:
        st.ctx.paged_evict(st.weights, st.pool, st.block_table, st.lengths, st.keep, st.weights_out, st.lengths_out, st.kept,
                           sinks=case["sinks"], recent=case["recent"])
        st.ctx.release_pages(st.lengths, st.lengths_out, st.block_table, st.queue, st.queue_state, st.queue_state_out, num_blocks=st.blocks)
    else:
        bsz, hkv, n = st.weights.shape
        pos, length = torch.arange(n, device="cuda"), st.lengths.long()[:, None, None]
        keep = torch.minimum(st.keep.long()[:, None, None], length)
        last = torch.clamp(keep, max=case["recent"])
        lead = torch.clamp(keep - last, max=case["sinks"])
        # kept for certain, then by weight (the first of equal ones), then what is behind the end
        rank = torch.where(pos >= length, -1.0, torch.where((pos < lead) | (pos >= length - last), torch.inf, st.weights.double()))
        order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
        chosen = torch.zeros(bsz, hkv, n, dtype=torch.bool, device="cuda").scatter_(2, order, (pos < keep).expand(bsz, hkv, n))
        b, h, src = chosen.nonzero(as_tuple=True)  # ascending slots of each head
        dst = (chosen.cumsum(-1) - 1)[b, h, src]
        table = st.block_table.long()
        sb, db = table[b, src // PAGE], table[b, dst // PAGE]
        parts = _parts(case)
        _move(st.pool, *parts[0], sb, src % PAGE, db, dst % PAGE, h)
        _move(st.pool, *parts[1], sb, src % PAGE, db, dst % PAGE, h)
        if case["bits"] < 16:
            _move(st.pool, *parts[-2], sb, src % PAGE, db, dst % PAGE, h)
            _move(st.pool, *parts[-1], sb, src % PAGE, db, dst % PAGE, h)
        if case["bits"] == 4:
            _move(st.pool, *parts[2], sb, src % PAGE, db, dst % PAGE, h)
            _move(st.pool, *parts[3], sb, src % PAGE, db, dst % PAGE, h)
        st.weights_out.copy_(torch.where(pos < length, 0.0, st.weights_out))
        st.weights_out[b, h, dst] = st.weights[b, h, src]
        st.kept[b, h, dst] = src.to(torch.int32)
        st.lengths_out.copy_(keep.flatten())
        # pages that hold no token any more go to the queue's end
        old, new = (st.lengths.long() + PAGE - 1) // PAGE, (keep.flatten() + PAGE - 1) // PAGE
        j = torch.arange(st.max_blocks, device="cuda")[None, :]
        head, count = st.queue_state.long()
        gone = (j >= new[:, None]) & (j < old[:, None])
        k = gone.flatten().cumsum(0).view(gone.shape) - 1
        cap = st.queue.numel()
        wide = torch.cat([st.queue, st.queue[:1]])
        wide[torch.where(gone, (head + count + k) % cap, cap).flatten()] = st.block_table.flatten()
        st.queue.copy_(wide[:cap])
        st.queue_state_out.copy_(torch.stack([head, count + gone.sum()]))
    return {"pool": _pool_views(case, st.pool), "weights": st.weights_out, "kept": st.kept, "lengths": st.lengths_out, "queue": st.queue,
            "queue_state": st.queue_state_out}


# ---------------------------------------------------------------- what a pass cannot do without
def _vector_bytes(case):
    """Bytes of a token's key (or value) of one head."""
    return _tile_bytes(case["bits"], case["d"]) / (2 * PAGE)


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "store":
        return {"bytes": 2 * case["tokens"] * hkv * (2 * d + _vector_bytes(case)) + 8 * (case["tokens"] + case["pad"]), "flops": 0}
    lens = _lengths(case)
    if case["op"] == "evict":
        keep = [min(n, case["keep"]) for n in lens]
        # tokens in front of the first one that goes stay where they are; the others move
        moved = sum(max(0, k - case["sinks"]) for n, k in zip(lens, keep) if k < n)
        pages = sum((n + PAGE - 1) // PAGE - (k + PAGE - 1) // PAGE for n, k in zip(lens, keep))
        return {"bytes": hkv * (8 * sum(lens) + 4 * sum(keep) + 4 * moved * _vector_bytes(case)) + 8 * pages + 12 * case["batch"], "flops": 0}
    seen = sum(min(n, case["window"]) if case["window"] else n for n in lens)
    table = 4 * sum((n + PAGE - 1) // PAGE for n in lens)
    rows = case["batch"] * case["hq"]
    if case["op"] == "weights":
        return {"bytes": hkv * (seen * _vector_bytes(case) + 8 * sum(lens)) + table + rows * (2 * d + 4) + 4 * case["batch"],
                "flops": 2.0 * seen * case["hq"] * d}
    return {"bytes": seen * hkv * 2 * _vector_bytes(case) + table + rows * (d * 6 + 4) + 4 * case["batch"], "flops": 4.0 * seen * case["hq"] * d}


# ---------------------------------------------------------------- the definitions in 64 bits
def _power(e):
    """2^e in 64 bits for whole e, without a rounding."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e2m1(c):
    """Values of 4-bit codes: a sign, two exponent bits (bias 1), one fraction bit."""
    c = c.to(torch.int64)
    e, f = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, 0.5 * f, (1.0 + 0.5 * f) * _power(e - 1))
    return torch.where(c >= 8, -v, v)


def _exact_rows(case, st, b, h):
    """Keys and values [tokens, d] in 64 bits of one head of one sequence."""
    d, n = case["d"], _lengths(case)[b]
    p = torch.arange(n, device="cuda")
    tile, t = st.pool[st.block_table[b].long()[p // PAGE], h], p % PAGE
    i = torch.arange(n, device="cuda")
    row = case["bits"] * d // 8
    raw = tile[:, :2 * PAGE * row].unflatten(1, (2, PAGE, row))[i, :, t]  # [tokens, 2, row]
    if case["bits"] == 16:
        x = raw.contiguous().view(DTYPES[case["dtype"]]).double()
    elif case["bits"] == 8:
        x = raw.contiguous().view(torch.float8_e4m3fn).double()
    else:
        x = torch.stack([_e2m1(raw & 15), _e2m1(raw >> 4)], -1).flatten(-2)
        s = tile[:, 16 * d:18 * d].unflatten(1, (2, PAGE, d // BLOCK))[i, :, t].contiguous().view(torch.float8_e4m3fn).double()
        x = x * s.repeat_interleave(BLOCK, -1)
    if case["bits"] < 16:
        x = x * _power(tile[:, -2 * PAGE:].unflatten(1, (2, PAGE))[i, :, t].view(torch.int8))[..., None]
    return x[:, 0], x[:, 1]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "store":
        return _exact_store(case, st)
    if case["op"] == "evict":
        return _exact_evict(case, st)
    bsz, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    rep = hq // hkv
    attend = case["op"] == "attend"
    out = torch.zeros(bsz, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((bsz, hq), -math.inf, dtype=torch.float64, device="cuda")
    weights = st.weights_out.double() if not attend else None
    for b, n in enumerate(_lengths(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        back = torch.arange(lo - n + 1, 1, device="cuda").double()
        for h in range(hkv):
            k, v = _exact_rows(case, st, b, h)
            if not attend:
                weights[b, h, :n] = case["decay"] * st.weights[b, h, :n].double()
            for g in range(h * rep, (h + 1) * rep):
                s = (k[lo:] * st.q[b, g].double()).sum(1) / math.sqrt(d)
                if case["cap"]:
                    s = case["cap"] * torch.tanh(s / case["cap"])
                if case["slopes"]:
                    s = s + st.slopes[g].double() * back
                if attend:
                    lse[b, g] = torch.logsumexp(s, 0)
                    out[b, g] = (torch.exp(s - lse[b, g])[:, None] * v[lo:]).sum(0)
                else:
                    weights[b, h, lo:n] += torch.exp(s - st.lse[b, g].double())
    return {"out": out, "lse": lse} if attend else weights


def _exact_store(case, st):
    """Block scales in 64 bits; codes and exponents are whole numbers."""
    d = case["d"]
    scales = st.pool[..., 16 * d:18 * d].view(torch.float8_e4m3fn).double().unflatten(-1, (2, PAGE, d // BLOCK))
    for i, x in enumerate((st.k, st.v)):
        x = x[:case["tokens"]].double()
        top = x.abs().amax(2, keepdim=True)
        e = torch.full_like(top, -120, dtype=torch.int64)
        for k in range(-120, 120):  # the least e with top <= 2688 * 2^e
            e = torch.where(top > 2688.0 * 2.0 ** k, k + 1, e)
        s = (x / _power(e)).unflatten(2, (-1, BLOCK)).abs().amax(-1) / 6.0
        step = torch.full_like(s, 2.0 ** -9)  # rounded to 3 fraction bits (ties to even), at least a multiple of 2^-9
        for k in range(-6, 9):
            step = torch.where(s >= 2.0 ** k, 2.0 ** (k - 3), step)
        slot = st.slots[:case["tokens"]]
        scales[slot // PAGE, :, i, slot % PAGE] = torch.round(s / step) * step
    return {"codes": None, "scales": scales.flatten(2), "exponents": None}


def _exact_evict(case, st):
    """The sums of the tokens that stay; everything else is moved as it is."""
    out = st.weights_out.double()
    for b, n in enumerate(_lengths(case)):
        keep = min(case["keep"], n)
        last = min(case["recent"], keep)
        lead = min(case["sinks"], keep - last)
        for h in range(case["hkv"]):
            w = st.weights[b, h, :n].double().cpu().numpy()
            p = np.arange(lead, n - last)
            free = p[np.lexsort((p, -w[lead:n - last]))][:keep - last - lead]
            stay = np.concatenate([np.arange(lead), np.sort(free), np.arange(n - last, n)])
            out[b, h, :n] = 0.0
            out[b, h, :keep] = torch.from_numpy(w[stay]).cuda()
    return {"pool": None, "weights": out, "kept": None, "lengths": None, "queue": None, "queue_state": None}
