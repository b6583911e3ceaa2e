"""CPU oracle of what a rollout and a training step run around the linear layers: the backward pass of the RMS norm, rotary
positions, the units that share a prompt, forks and sweeps of the key/value cache.

TEST INFRASTRUCTURE ONLY: imported by tests/.  The product library never imports it.

Source: Jet-RL explainers, "Enonce du Probleme" (rollout of several samples is most of RL training time) and "Schema de
Quantification" (gradients between operators stay BF16).  The pages give no such operators; the definitions are those of
include/jetfp8.h, computed here in float64 and in plain loops over requests, units and table entries.
"""
import numpy as np

BLOCK, SPAN = 64, 8


def rmsnorm_backward(dy, h, w, rstd, dres=None):
    """float64 arrays (rstd the fp32 values) -> dx, dw and bounds on the error of an fp32 computation of them, before dx is
    rounded to bf16.  A row's sum has at most 43 roundings in line (32 products of a lane, 6 exchanges, 5 waves), the rest
    of dx 5; a column's sum one for each of a team's rows (at most ceil(rows / 1024), no team has more) and 5 others."""
    R, C = h.shape
    r = rstd[:, None]
    g = dy * w
    mean = (g * h).sum(1, keepdims=True) / C
    dx = r * (g - h * r * r * mean)
    u = 2.0 ** -24
    size = np.abs(r * g) + np.abs(r ** 3 * h * mean)
    bound = 6 * u * size + 48 * u * np.abs(r ** 3 * h) * np.abs(g * h).sum(1, keepdims=True) / C
    if dres is not None:
        dx = dx + dres
        bound += 2 * u * np.abs(dres)
    terms = dy * h * r
    dw = terms.sum(0)
    return dx, bound + 2.0 ** -133, dw, ((-(-R // 1024) + 5) * u) * np.abs(terms).sum(0) + 2.0 ** -140


def rotary(x, positions, freqs, interleaved, amplitude, inverse):
    """x float64 [T, heads, D] -> the turned values, and a bound on the error of cosines, sines and products in fp32: the
    argument in half turns, its cosine or sine (2 steps) and the amplitude's product are off by less than 2^-22 of 1, and a
    pair's two products and their sum by 2^-23 of |a| + |b|."""
    P = len(freqs)
    out, bound = x.copy(), np.zeros_like(x)
    i = np.arange(P)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, P + i)
    angle = (positions.astype(np.float64)[:, None] * freqs)[:, None, :] * (-1 if inverse else 1)
    c, s = amplitude * np.cos(angle), amplitude * np.sin(angle)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    bound[..., a] = bound[..., b] = amplitude * (np.abs(x[..., a]) + np.abs(x[..., b])) * 2.0 ** -21 + 2.0 ** -140
    idle = positions < 0
    out[idle], bound[idle] = np.nan, np.nan
    return out, bound


def positions(units, tokens):
    out = np.full(tokens, -1, np.int32)
    for r, j, _, row, rows, offset, _, _ in units:
        if r >= 0:
            out[row:row + rows] = j * BLOCK + offset + np.arange(rows)
    return out


def prefix(units, table, groups):
    """Records of the units, one group after the other."""
    out = np.zeros((len(units), 4), np.int32)
    for k, u in enumerate(units):
        out[k, :2] = (k, 1) if u[0] >= 0 else (-1, 0)
    R, start = len(groups), 0
    while start < R:
        end = start + 1
        while groups[start] >= 0 and end < R and groups[end] == groups[start]:
            end += 1
        mine = [k for k, u in enumerate(units) if start <= u[0] < end]
        live = sorted({int(units[k][0]) for k in mine})
        if groups[start] >= 0 and len(live) > 1:
            common = min(int(units[k][1]) for k in mine)
            common = min(common, table.shape[1])
            for r in live[1:]:
                n = 0
                while n < common and table[r, n] == table[live[0], n]:
                    n += 1
                common = n
            common = common // SPAN * SPAN
            if common:
                for k in mine:
                    out[k] = mine[0], len(mine), common, 0
        start = end
    return out


def parent(parents, state, r):
    p = int(parents[r])
    fits = 0 <= p < len(parents) and state[r, 1] in (0, 1) and state[p, 1] in (0, 1)
    return p if fits else r


def fork(state, table, parents):
    next_state, next_table = state.copy(), np.full_like(table, -1)
    for r in range(len(state)):
        p = parent(parents, state, r)
        held = min(max(int(state[p, 0]), 0) // BLOCK, table.shape[1])
        next_table[r, :held] = table[p, :held]
        if p != r:
            next_state[r] = state[p, 0], 1 - state[r, 1]
    return next_state, next_table


def fork_recent(parents, state, recent):
    """Changed in place; the parents' blocks are those before the call."""
    old = recent.copy()
    for r in range(len(state)):
        p = parent(parents, state, r)
        if p != r:
            recent[2 * r + 1 - state[r, 1]] = old[2 * p + state[p, 1]]


def sweep(state, table, num_blocks, compact):
    """free_blocks, free_head, live and, with compact, next_table and moves."""
    held = [min(max(int(n), 0) // BLOCK, table.shape[1]) for n in state[:, 0]]
    live = {int(b) for row, n in zip(table, held) for b in row[:n] if 0 <= b < num_blocks}
    L = len(live)
    free = [b for b in range(num_blocks) if (b >= L if compact else b not in live)]
    out = dict(free_blocks=np.array(free + [-1] * (num_blocks - len(free)), np.int32), free_head=np.zeros(1, np.int32),
               live=np.array([L], np.int32), next_table=None, moves=None)
    if compact:
        source = sorted(b for b in live if b >= L)
        target = [b for b in range(L) if b not in live]
        to = dict(zip(source, target))
        out["moves"] = np.full((max(1, num_blocks // 2), 2), -1, np.int32)
        out["moves"][:len(to)] = np.array(list(to.items()), np.int32).reshape(-1, 2)
        out["next_table"] = np.full_like(table, -1)
        for r, n in enumerate(held):
            for j in range(n):
                b = int(table[r, j])
                out["next_table"][r, j] = to.get(b, b) if 0 <= b < num_blocks else -1
    return out
