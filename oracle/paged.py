"""Page plan, dense-layout pages and their single-token attention, in float64 and Python integers.

Pages hold 16 tokens.  A 16-bit tile is keys [16][d] then values [16][d]; an 8-bit tile is key codes
[16][d], value codes [16][d] (e4m3), then int8 exponents of the keys and of the values; a 4-bit tile is key codes
[16][d / 2], value codes [16][d / 2] (e2m1, entry 2 i in the low half of byte i), e4m3 scales of 16 entries [16][d / 16]
of the keys and of the values, then the exponents.
"""
import numpy as np

PAGE, RING = 16, 128
ERR_BLOCK_ID, ERR_POSITION, ERR_PAGES = 0x1, 0x2, 0x20


# ---------------------------------------------------------------- number formats
def to_f64(bits16, bf16):
    """float64 of fp16 or bf16 bit patterns."""
    b = np.asarray(bits16, np.uint16)
    if bf16:
        return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return b.view(np.float16).astype(np.float64)


def e4m3_value(code):
    """float64 of e4m3 codes: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7f is NaN, no infinities."""
    c = np.asarray(code, np.uint8).astype(np.int64)
    s = np.where(c & 0x80, -1.0, 1.0)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    return np.where((c & 0x7F) == 0x7F, np.nan, s * v)


_POS = e4m3_value(np.arange(0x7F))  # the non-negative values, ascending


def e4m3_code(x):
    """Codes of float64 values: nearest, ties to the even code; beyond 448 saturates, NaN is 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.searchsorted(_POS, a).clip(0, len(_POS) - 1)
    lo = (hi - 1).clip(0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.signbit(x), c | 0x80, c)
    return np.where(np.isnan(x), (c & 0x80) | 0x7F, c).astype(np.uint8)


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_value(code):
    """float64 of e2m1 codes: sign, 2 exponent bits (bias 1), 1 fraction bit."""
    c = np.asarray(code, np.uint8)
    return np.where(c & 8, -E2M1[c & 7], E2M1[c & 7])


def e2m1_code(x):
    """Codes of float64 values: nearest, ties to the even code, beyond 6 saturates; the sign is x's."""
    x = np.asarray(x, np.float64)
    d = np.abs(np.minimum(np.abs(x), 6.0)[..., None] - E2M1)
    best = d.min(-1)
    lo = np.argmax(d == best[..., None], -1)
    c = np.where((np.take_along_axis(d, np.minimum(lo + 1, 7)[..., None], -1)[..., 0] == best) & (lo % 2 == 1) & (lo < 7), lo + 1, lo)
    return np.where(np.signbit(x), c | 8, c).astype(np.uint8)


def quantise4(x):
    """(codes [d], scale codes [d / 16], e) of a vector of float64."""
    e = int(exponent(x, 2688.0))
    y = (x * 2.0 ** -e).reshape(-1, 16)
    a = np.abs(y)
    scale = e4m3_code(np.where(np.isfinite(a), a, 0.0).max(-1) / 6.0)
    scale = np.where(np.isinf(a).any(-1), 0x7E, scale)
    nan = np.isnan(a).any(-1)
    s = e4m3_value(scale)[:, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s > 0, y / s, np.copysign(0.0, y))
    codes = np.where(nan[:, None], 0, e2m1_code(np.where(np.isnan(q), 0.0, q)))
    return codes.reshape(-1).astype(np.uint8), np.where(nan, 0x7F, scale).astype(np.uint8), e


def exponent(x, most=448.0):
    """e = least whole number >= -120 with max|x| <= most * 2^e over the finite entries of the last axis."""
    a = np.abs(np.asarray(x, np.float64))
    top = np.where(np.isfinite(a), a, 0.0).max(-1)
    e = np.full(top.shape, -120)
    for k in range(-120, 121):
        e = np.where(top > most * 2.0 ** k, k + 1, e)
    return e


# ---------------------------------------------------------------- tiles
def tile_bytes(d, bits):
    return 64 * d if bits == 16 else 32 * d + 32 if bits == 8 else 18 * d + 32


def tile_rows(tile, d, bits, bf16):
    """(keys, values) float64 [16][d] of one tile."""
    t = np.ascontiguousarray(tile)
    if bits == 16:
        x = to_f64(t.view(np.uint16), bf16).reshape(2, PAGE, d)
    elif bits == 4:
        e = t[18 * d:].view(np.int8).astype(np.float64).reshape(2, PAGE, 1)
        c = np.stack([t[:16 * d] & 15, t[:16 * d] >> 4], -1).reshape(2, PAGE, d)
        x = e2m1_value(c) * np.repeat(e4m3_value(t[16 * d:18 * d]).reshape(2, PAGE, d // 16), 16, -1) * 2.0 ** e
    else:
        e = t[32 * d:].view(np.int8).astype(np.float64).reshape(2, PAGE, 1)
        x = e4m3_value(t[:32 * d]).reshape(2, PAGE, d) * 2.0 ** e
    return x[0], x[1]


def store(pool, k16, v16, slots, d, bits, bf16):
    """Write rows (bit patterns [n][hkv][d]) into a copy of pool; returns (pool, error flags)."""
    pool, flags = pool.copy(), 0
    for i, slot in enumerate(slots):
        if slot < 0:
            continue
        block, t = int(slot) // PAGE, int(slot) % PAGE
        if block >= pool.shape[0]:
            flags |= ERR_BLOCK_ID
            continue
        for h in range(pool.shape[1]):
            tile = pool[block, h]
            for side, x in enumerate((k16[i, h], v16[i, h])):
                at = side * PAGE + t
                if bits == 16:
                    tile[2 * d * at:2 * d * (at + 1)] = np.ascontiguousarray(x).view(np.uint8)
                elif bits == 4:
                    c, s, e = quantise4(to_f64(x, bf16))
                    tile[d // 2 * at:d // 2 * (at + 1)] = c[0::2] | c[1::2] << 4
                    tile[16 * d + d // 16 * at:16 * d + d // 16 * (at + 1)] = s
                    tile[18 * d + at] = e & 0xFF
                else:
                    f = to_f64(x, bf16)
                    e = int(exponent(f))
                    tile[d * at:d * (at + 1)] = e4m3_code(f * 2.0 ** -e)
                    tile[32 * d + at] = e & 0xFF
    return pool, flags


# ---------------------------------------------------------------- attention
def attention(q, pool, block_table, lengths, d, bits, bf16, window=0, scale=None, cap=0.0, slopes=None, weights=None):
    """q float64 [batch][hq][d] -> (out, lse, reach, flags); reach [batch][hq] = (max_p sum_i |scale q_i k_pi|,
    sum_p p |v| over the weights), the magnitudes a rounding bound needs: reach is (a, vabs [.., d]).  Scores are capped by
    cap * tanh(. / cap) and biased by slopes[h] * (position - newest position); weights, a list, receives per sequence and head
    (positions, scores, sum_i |scale q_i k_pi| + |slope (p - newest)|)."""
    bsz, hq, _ = q.shape
    hkv = pool.shape[1]
    rep = hq // hkv
    scale = 1.0 / np.sqrt(d) if not scale else scale
    out, lse = np.zeros((bsz, hq, d)), np.full((bsz, hq), -np.inf)
    reach_s, reach_v, flags = np.zeros((bsz, hq)), np.zeros((bsz, hq, d)), 0
    for b in range(bsz):
        n = int(lengths[b])
        if n < 0 or n > block_table.shape[1] * PAGE:
            flags |= ERR_POSITION
            continue
        lo = max(0, n - window) if window else 0
        ks, vs, ps = [], [], []
        for pg in range(lo // PAGE, -(-n // PAGE)):
            block = int(block_table[b, pg])
            if block < 0 or block >= pool.shape[0]:
                flags |= ERR_BLOCK_ID
                continue
            t0, t1 = max(lo - pg * PAGE, 0), min(n - pg * PAGE, PAGE)
            kv = [tile_rows(pool[block, h], d, bits, bf16) for h in range(hkv)]
            ks.append(np.stack([x[0][t0:t1] for x in kv]))
            vs.append(np.stack([x[1][t0:t1] for x in kv]))
            ps.append(np.arange(pg * PAGE + t0, pg * PAGE + t1))
        if not ks:
            continue
        k, v, p_at = np.concatenate(ks, 1), np.concatenate(vs, 1), np.concatenate(ps)  # [hkv][n][d]
        for h in range(hq):
            s = scale * (k[h // rep] @ q[b, h])
            reach = abs(scale) * (np.abs(k[h // rep]) @ np.abs(q[b, h]))
            if cap:
                s = cap * np.tanh(s / cap)
            if slopes is not None:
                s = s + slopes[h] * (p_at - (n - 1))
                reach = reach + np.abs(slopes[h] * (p_at - (n - 1)))
            if weights is not None:
                weights.append((b, h, p_at, s, reach))
            m = s.max()
            p = np.exp(s - m)
            out[b, h] = p @ v[h // rep] / p.sum()
            lse[b, h] = m + np.log(p.sum())
            reach_s[b, h] = np.max(reach)
            reach_v[b, h] = p @ np.abs(v[h // rep]) / p.sum()
    return out, lse, (reach_s, reach_v), flags


def weight_sums(q, pool, block_table, lengths, lse, before, decay, d, bits, bf16, window=0, scale=None, cap=0.0, slopes=None):
    """(sums [batch][hkv][n], bound factor: the largest reach of each entry, flags) of before [batch][hkv][n]."""
    rep, out, seen = q.shape[1] // pool.shape[1], np.array(before, np.float64), []
    reach = np.zeros_like(out)
    lens, flags = np.array(lengths).copy(), 0
    for b, n in enumerate(lens):
        if n < 0 or n > min(block_table.shape[1] * PAGE, out.shape[2]):
            lens[b], flags = 0, ERR_POSITION
        out[b, :, :lens[b]] *= decay
    flags |= attention(q, pool, block_table, lens, d, bits, bf16, window, scale, cap, slopes, seen)[3]
    for b, h, p, s, r in seen:
        if lse[b, h] != -np.inf:
            out[b, h // rep, p] += np.exp(s - lse[b, h])
        reach[b, h // rep, p] = np.maximum(reach[b, h // rep, p], r)
    return out, reach, flags


# ---------------------------------------------------------------- eviction
def choose(weights, keep, sinks, recent):
    """The slots that stay of a row of weights, ascending."""
    n = len(weights)
    keep = max(min(keep, n), 0)
    last = min(recent, keep)
    lead = min(sinks, keep - last)
    between = sorted(range(lead, n - last), key=lambda p: (0, p) if np.isnan(weights[p]) else (1, -weights[p], p))
    return sorted(list(range(lead)) + between[:keep - last - lead] + list(range(n - last, n)))


def token_bytes(tile, t, d, bits):
    """Views of the parts of a tile that hold token t's key and value."""
    row = d * bits // 8
    parts = [tile[s * PAGE * row + t * row:s * PAGE * row + (t + 1) * row] for s in (0, 1)]
    at = 2 * PAGE * row
    if bits == 4:
        parts += [tile[at + (s * PAGE + t) * (d // 16):at + (s * PAGE + t + 1) * (d // 16)] for s in (0, 1)]
        at += 2 * d
    if bits < 16:
        parts += [tile[at + s * PAGE + t:at + s * PAGE + t + 1] for s in (0, 1)]
    return parts


def evict(weights, pool, block_table, lengths, keep, sinks, recent, d, bits):
    """dict(pool, lengths, kept: list of lists, weights: list of lists, flags); pool is a copy."""
    pool, flags = pool.copy(), 0
    old, kept_all, lens, sums = pool.copy(), [], [], []
    for b in range(len(lengths)):
        n = int(lengths[b])
        if n < 0 or n > min(block_table.shape[1] * PAGE, weights.shape[2]):
            n, flags = 0, flags | ERR_POSITION
        kept_all.append([])
        sums.append([])
        for h in range(pool.shape[1]):
            kept = choose(weights[b, h, :n], int(keep[b]), sinks, recent)
            for i, p in enumerate(kept):
                if i == p:
                    continue
                src, dst = int(block_table[b, p // PAGE]), int(block_table[b, i // PAGE])
                if not (0 <= src < pool.shape[0] and 0 <= dst < pool.shape[0]):
                    flags |= ERR_BLOCK_ID
                    continue
                for x, y in zip(token_bytes(pool[dst, h], i % PAGE, d, bits), token_bytes(old[src, h], p % PAGE, d, bits)):
                    x[:] = y
            kept_all[b].append(kept)
            sums[b].append(np.concatenate([weights[b, h, kept], np.zeros(n - len(kept), weights.dtype)]))
        lens.append(len(kept_all[b][0]))
    return dict(pool=pool, lengths=np.array(lens, np.int32), kept=kept_all, weights=sums, flags=flags)


def release(lengths, new_lengths, block_table, queue, queue_state, num_blocks):
    """(queue, queue_state, flags) with the pages that hold nothing any more."""
    queue, flags, cap = queue.copy(), 0, len(queue)
    head, count = int(queue_state[0]), int(queue_state[1])
    if not (0 <= count <= cap and 0 <= head and (head < cap or cap == 0)):
        return queue, queue_state.copy(), ERR_PAGES | (ERR_POSITION if any(
            not 0 <= m <= n <= block_table.shape[1] * PAGE for n, m in zip(lengths, new_lengths)) else 0)
    for b, (n, m) in enumerate(zip(lengths, new_lengths)):
        if not 0 <= m <= n <= block_table.shape[1] * PAGE:
            flags |= ERR_POSITION
            continue
        for j in range(-(-int(m) // PAGE), -(-int(n) // PAGE)):
            if count == cap:
                flags |= ERR_PAGES
                continue
            queue[(head + count) % cap] = block_table[b, j]
            flags |= 0 if 0 <= block_table[b, j] < num_blocks else ERR_BLOCK_ID
            count += 1
    return queue, np.array([head, count], np.int32), flags


# ---------------------------------------------------------------- plan
def pages_of(tokens, ring):
    if ring:
        return max(tokens - 1, 0) // RING * (RING // PAGE)
    return -(-tokens // PAGE)


def plan(ctx_len, new_len, block_table, queue, queue_state, num_blocks, max_tokens, ring=0):
    """One step's page plan; returns a dict of the outputs and the error flags."""
    bsz, maxb, cap = len(ctx_len), block_table.shape[1], len(queue)
    table, q_out, flags = block_table.copy(), queue.copy(), 0
    head, count = int(queue_state[0]), int(queue_state[1])
    sound_queue = 0 <= count <= cap and 0 <= head and (head < cap or cap == 0)
    if not sound_queue:
        flags |= ERR_PAGES
        head = count = 0
    lengths, paged, starts = np.zeros(bsz, np.int32), np.zeros(bsz, np.int32), np.zeros(bsz + 1, np.int32)
    slots = np.full(max_tokens, -1, np.int64)
    positions, rows = np.full(max_tokens, -1, np.int32), np.full(max_tokens, -1, np.int32)
    tok = wanted = taken = back = 0
    room = cap - count if sound_queue else 0
    for b in range(bsz):
        c, n = int(ctx_len[b]), int(new_len[b])
        ended, add = n < 0, max(n, 0)
        starts[b] = tok
        total = c + add
        sound = c >= 0 and pages_of(total, ring) <= maxb and total < 2 ** 31
        if not sound:
            flags |= ERR_POSITION
        old = pages_of(max(c, 0), ring)
        need = pages_of(total, ring) - old if sound and not ended else 0
        ok = sound and (add == 0 or tok + add <= max_tokens) and (need == 0 or wanted + need <= count)
        if sound and not ok:
            flags |= ERR_PAGES
        length = 0 if ended else total if ok else max(c, 0)
        lengths[b] = length
        paged[b] = max(length - 1, 0) // RING * RING if ring else length
        if ok and need:
            for j in range(need):
                i = int(queue[(head + wanted + j) % cap])
                if not 0 <= i < num_blocks:
                    i, flags = -1, flags | ERR_BLOCK_ID
                table[b, old + j] = i
            taken = wanted + need
        if ended and sound:
            for j in range(old):
                if back < room:
                    q_out[(head + count + back) % cap] = block_table[b, j]
                    if not 0 <= block_table[b, j] < num_blocks:
                        flags |= ERR_BLOCK_ID
                    back += 1
                else:
                    flags |= ERR_PAGES
        for i in range(add):
            if tok + i >= max_tokens:
                break
            p = c + i
            positions[tok + i], rows[tok + i] = (p if c >= 0 and p < 2 ** 31 else -1), b
            if ok and p < paged[b]:
                block = int(table[b, p // PAGE])
                if 0 <= block < num_blocks:
                    slots[tok + i] = block * PAGE + p % PAGE
                else:
                    flags |= ERR_BLOCK_ID
        tok += add
        wanted += need
    starts[bsz] = tok
    state = np.array([(head + taken) % cap if cap else 0, count - taken + back] if sound_queue else queue_state, np.int32)
    return dict(block_table=table, queue=q_out, queue_state=state, lengths=lengths, n_paged=paged, n_ring=lengths - paged,
                token_start=starts, slots=slots, positions=positions, rows=rows, flags=flags)
