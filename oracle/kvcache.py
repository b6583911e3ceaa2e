"""CPU oracle of the FP8 key/value cache: the step's plan, the append of keys and values, and the attention.

TEST INFRASTRUCTURE ONLY: imported by tests/.  The product library never imports it.

Source: Jet-RL explainers, "Architecture Centrale" (rollout and the training forward share one graph and one
quantization) and "Schema de Quantification" (dynamic group scales).  The pages give no cache; the definitions are
those of include/jetfp8.h, computed here one request, block and head at a time in plain integer and float64 loops:

  * block j of a request holds its positions 64 j .. 64 j + 63; complete, it is E4M3 with s = fl32(amax / 448) over
    the 64 x D keys (values) of a kv head, codes the nearest E4M3 values to x / s, ties to the even code;
  * a query at position t reads blocks before t // 64 as code * scale, its own block's positions up to t as bf16;
  * o = sum softmax(scale * q . k) v.
"""
import numpy as np

from . import decode

BLOCK = 64
BAD_LENGTH, NO_ROWS, NO_BLOCK = 1, 2, 4
E4M3 = np.array([decode(c) for c in range(256)])
_POS = E4M3[:127]
_MID = (_POS[1:] + _POS[:-1]) / 2


def e4m3_codes(z) -> np.ndarray:
    """Nearest E4M3 codes of float64 values, ties to the even code, magnitudes beyond 448 saturated."""
    a = np.abs(z)
    i = np.searchsorted(_MID, a, side="left")               # _MID[i - 1] < a <= _MID[i]
    tie = (i < 126) & (a == _MID[np.minimum(i, 125)]) & (i % 2 == 1)
    return (i + tie + np.where(np.signbit(z), 128, 0)).astype(np.uint8)


def quantize_block(x):
    """x float64 (bf16 values) of one block and head -> codes of the same shape, scale (np.float32)."""
    s = np.float32(np.abs(x).max()) / np.float32(448)
    if s == 0:
        return np.where(np.signbit(x), 128, 0).astype(np.uint8), s
    return e4m3_codes(x / np.float64(s)), s


def places(D):
    """[64, D] places of key n, channel d in a block's memory: E4M3 keys, E4M3 values, bf16 keys, bf16 values."""
    k8, v8, k16, v16 = (np.empty((BLOCK, D), dtype=np.int64) for _ in range(4))
    for n in range(BLOCK):
        for d in range(D):
            k8[n, d] = ((n // 16 * (D // 64) + d // 64) * 64 + d % 32 // 8 * 16 + n % 16) * 16 + d % 64 // 32 * 8 + d % 8
            v8[n, d] = (d // 16 * 64 + n % 16 // 4 * 16 + d % 16) * 16 + n // 32 * 8 + n % 32 // 16 * 4 + n % 4
            k16[n, d] = ((n // 16 * (D // 32) + d // 32) * 64 + d % 32 // 8 * 16 + n % 16) * 8 + d % 8
            v16[n, d] = ((d // 16 * 2 + n // 32) * 64 + n % 16 // 4 * 16 + d % 16) * 8 + n % 32 // 16 * 4 + n % 4
    return k8, v8, k16, v16


def max_units(tokens, requests):
    return min(tokens, (tokens + 62 * requests) // BLOCK + requests)


def plan(state, new_lens, free_blocks, free_head, table, tokens, max_new, num_blocks=2 ** 31 - 1):
    """One request after the other.  Returns next_state, next_free, status, units, slots and the new table."""
    R, width = table.shape
    table, next_state = table.copy(), state.copy()
    status = np.zeros(R, dtype=np.int32)
    slots = np.full(tokens, -1, dtype=np.int64)
    units, row, middle, stopped = [], 0, 0, False
    head = start = min(max(int(free_head), 0), len(free_blocks))
    end = next((i for i in range(head, len(free_blocks)) if not 0 <= free_blocks[i] < num_blocks), len(free_blocks))
    for r in range(R):
        ctx, slot, n = int(state[r, 0]), int(state[r, 1]), int(new_lens[r])
        row += min(max(n, 0), tokens + 1)
        if ctx < 0 or n < 0 or n > max_new or ctx + n > BLOCK * width or slot not in (0, 1):
            status[r] = BAD_LENGTH
            continue
        if row > tokens:
            status[r] = NO_ROWS
            continue
        if n == 0:
            continue
        done = range(ctx // BLOCK, (ctx + n) // BLOCK)       # blocks that this step completes
        if len(done) and (stopped or head + len(done) > end):
            status[r], stopped = NO_BLOCK, True
            continue
        taken = {j: int(free_blocks[head + i]) for i, j in enumerate(done)}
        head += len(done)
        first, last = ctx // BLOCK, (ctx + n - 1) // BLOCK
        for j in range(first, last + 1):
            lo, hi = max(ctx, j * BLOCK), min(ctx + n, (j + 1) * BLOCK)
            if j == first:
                recent = 2 * r + slot
            elif j == last:
                recent = 2 * r + 1 - slot
            else:
                recent, middle = 2 * R + middle, middle + 1
            begin = row - n + lo - ctx
            units.append((r, j, recent, begin, hi - lo, lo - j * BLOCK, taken.get(j, -1), 0))
            if j in taken:
                table[r, j] = taken[j]
                slots[begin:begin + hi - lo] = taken[j] * BLOCK + lo - j * BLOCK + np.arange(hi - lo)
        next_state[r] = ctx + n, (slot if first == last else 1 - slot)
    out = np.full((max_units(tokens, R), 8), -1, dtype=np.int32)
    out[:len(units)] = np.array(units, dtype=np.int32).reshape(-1, 8)
    assert len(units) <= len(out) and start <= head
    return dict(next_state=next_state, next_free=np.array([head], dtype=np.int32), status=status, units=out,
                slots=slots, table=table)


def append(k, v, units, codes, scales, recent):
    """k, v: bf16 bits uint16 [T, H, D]; codes uint8, scales fp32 and recent uint16 bits are changed in place."""
    H, D = k.shape[1:]
    k8, v8, k16, v16 = places(D)
    for r, j, place, row, rows, offset, physical, _ in units:
        if r < 0:
            continue
        for h in range(H):
            for which, src, at8, at16 in ((0, k, k8, k16), (1, v, v8, v16)):
                block = recent[place, h, which]
                if offset == 0:
                    block[:] = 0
                for i in range(rows):
                    block[at16[offset + i]] = src[row + i, h]
                if physical >= 0:
                    x = bf16(block[at16])
                    c, s = quantize_block(x)
                    codes[physical, h, which][at8] = c
                    scales[physical, h, which] = s


def bf16(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def attention(q, units, table, codes, scales, recent, softmax_scale):
    """q float64 [T, Hq, D] -> o [T, Hq, D] (NaN where no unit has the row), and per output a bound on the error of a
    computation in fp32 whose probabilities are rounded to 11 bits (before the rounding of the result):
        |v| weighted by the probabilities * (2^-11 + 2 e + N 2^-22) + N 2^-31 * largest p_n * 448 s_n,
    2^-11 for the rounding of each probability; e for the relative error of an exponential, from the score's D products
    and sums, its scaling and the exponential itself; N 2^-22 for the sums over N keys.  The last term is for cached keys
    whose probability times their block's scale s_n is below 2^-20 of the largest such product of the row: those are
    subnormal in fp16.  It goes by what a block contributes to the row, so one without weight costs the others nothing."""
    T, Hq, D = q.shape
    H = codes.shape[1]
    G = Hq // H
    k8, v8, k16, v16 = places(D)
    out, bound = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for r, j, place, row, rows, offset, physical, _ in units:
        if r < 0:
            continue
        ids = [int(p) for p in table[r, :j] if 0 <= p < len(codes)]
        for h in range(H):
            K = [E4M3[codes[p, h, 0][k8]] * np.float64(scales[p, h, 0]) for p in ids]
            V = [E4M3[codes[p, h, 1][v8]] * np.float64(scales[p, h, 1]) for p in ids]
            weight = np.repeat([448 * np.float64(scales[p, h, 1]) for p in ids], BLOCK)
            own_k, own_v = bf16(recent[place, h, 0][k16]), bf16(recent[place, h, 1][v16])
            for i in range(rows):
                k = np.concatenate(K + [own_k[:offset + i + 1]])
                v = np.concatenate(V + [own_v[:offset + i + 1]])
                qs = q[row + i, h * G:(h + 1) * G]
                s = qs @ k.T * softmax_scale
                p = np.exp(s - s.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
                out[row + i, h * G:(h + 1) * G] = p @ v
                size = (np.abs(qs) @ np.abs(k).T).max(axis=1, keepdims=True) * softmax_scale
                e = (D + 8) * 2.0 ** -24 * size + 2.0 ** -21
                most = (p[:, :len(weight)] * weight).max(axis=1, keepdims=True) if ids else 0.0
                bound[row + i, h * G:(h + 1) * G] = (p @ np.abs(v)) * (2.0 ** -11 + 2 * e + len(k) * 2.0 ** -22) + \
                    len(k) * 2.0 ** -31 * most
    return out, bound
