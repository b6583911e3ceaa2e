"""The page operations of the key/value cache on the GPU against the oracle's loops, all whole numbers or copied bits:
positions, records of shared prompts, forks, sweeps and moves."""
import numpy as np
import pytest

from oracle import kvcache as kc
from oracle import rollout as ro

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jf():
    import torch
    import fp8_precision_rl_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.load_library()
    return m


def up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def plan(rng, R, ctx, new, width=None, idle=0.0):
    """A planned step of R requests: its oracle plan and the requests' state."""
    state = np.stack([rng.integers(0, ctx + 1, R), rng.integers(0, 2, R)], 1).astype(np.int32)
    lens = np.where(rng.random(R) < idle, 0, rng.integers(1, new + 1, R)).astype(np.int32)
    lens[0] = max(lens[0], 1)
    width = width or (ctx + new) // 64 + 1
    need = int(((state[:, 0] + lens) // 64 - state[:, 0] // 64).sum())
    table = rng.integers(0, 50, (R, width)).astype(np.int32)
    return kc.plan(state, lens, np.arange(1000, 1000 + need, dtype=np.int32), 0, table, int(lens.sum()) + 3, new), state


# ------------------------------------------------------------------------------------------------ positions, prefix
@pytest.mark.parametrize("R,ctx,new,idle", [(1, 0, 1, 0), (1, 70, 300, 0), (40, 500, 1, 0.3), (257, 90, 70, 0.2), (4096, 300, 3, 0.5)])
def test_positions(jf, R, ctx, new, idle):
    p, _ = plan(np.random.default_rng(R + new), R, ctx, new, idle=idle)
    T = int((p["units"][:, 4][p["units"][:, 0] >= 0]).sum())
    for tokens in (T, T + 3, 1, T + 5000):
        got = jf.kv_positions(up(p["units"]), tokens)
        want = ro.positions(p["units"], max(tokens, T))[:tokens]
        assert np.array_equal(got.cpu().numpy(), want)


def shared_tables(rng, R, width, sizes):
    """Tables of groups of the given sizes that agree in some leading blocks."""
    table = rng.integers(0, 5000, (R, width)).astype(np.int32)
    groups = np.full(R, -1, np.int32)
    r = 0
    for i, n in enumerate(sizes):
        n = min(n, R - r)
        if n == 0:
            break
        common = int(rng.choice([0, 3, 7, 8, 9, 15, 16, 63, 64, 65, width]))
        table[r:r + n, :common] = table[r, :common]
        if rng.random() < 0.8:
            groups[r:r + n] = i % 3 if rng.random() < 0.3 else i
        r += n
    return table, groups


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("R,ctx,new,idle", [(1, 900, 1, 0), (7, 5000, 1, 0.2), (40, 6000, 3, 0.3), (64, 700, 130, 0.3),
                                            (300, 9000, 1, 0.1), (1000, 2000, 2, 0.9)])
def test_prefix(jf, R, ctx, new, idle, seed):
    rng = np.random.default_rng(R + seed)
    p, _ = plan(rng, R, ctx, new, idle=idle)
    table, groups = shared_tables(rng, R, p["table"].shape[1], rng.integers(1, [3, 20, 300][seed % 3], R))
    got = jf.kv_prefix(up(p["units"]), up(table), up(groups))
    assert np.array_equal(got.cpu().numpy(), ro.prefix(p["units"], table, groups))


def test_prefix_one_group_of_all(jf):
    """The most requests, all alike: the longest scans."""
    rng = np.random.default_rng(5)
    R, width = 4096, 70
    state = np.stack([np.full(R, 64 * 66 + 5), np.zeros(R)], 1).astype(np.int32)
    table = np.tile(rng.integers(0, 100, width).astype(np.int32), (R, 1))
    p = kc.plan(state, np.ones(R, np.int32), np.zeros(0, np.int32), 0, table, R, 1)
    for break_at in (None, 64, 31):
        if break_at is not None:
            table[R - 1, break_at] = 7777
        want = ro.prefix(p["units"], table, np.zeros(R, np.int32))
        got = jf.kv_prefix(up(p["units"]), up(table), up(np.zeros(R, np.int32)))
        assert np.array_equal(got.cpu().numpy(), want) and want[0, 2] == {None: 64, 64: 64, 31: 24}[break_at]


# ------------------------------------------------------------------------------------------------ fork
@pytest.mark.parametrize("R,width", [(1, 1), (5, 3), (64, 20), (257, 300), (4096, 7)])
def test_fork(jf, R, width):
    rng = np.random.default_rng(R)
    state = np.stack([rng.integers(-5, 64 * width + 1, R), rng.integers(0, 2, R)], 1).astype(np.int32)
    state[rng.random(R) < 0.05, 1] = 2                                     # no recent block: they stay, and so do their copies
    table = rng.integers(-1, 10000, (R, width)).astype(np.int32)
    maps = [np.full(R, -1), np.arange(R), np.arange(R)[::-1], np.zeros(R), rng.integers(0, R, R), rng.integers(-2, R + 3, R)]
    for parents in maps:
        parents = parents.astype(np.int32)
        f = jf.kv_fork(up(state), up(table), up(parents))
        want = ro.fork(state, table, parents)
        assert np.array_equal(f.next_state.cpu().numpy(), want[0]) and np.array_equal(f.next_table.cpu().numpy(), want[1])


@pytest.mark.parametrize("R,H,D", [(1, 1, 64), (6, 3, 64), (9, 8, 128), (70, 2, 128)])
def test_fork_recent(jf, R, H, D):
    import torch
    rng = np.random.default_rng(R)
    state = np.stack([rng.integers(0, 500, R), rng.integers(0, 2, R)], 1).astype(np.int32)
    if R > 5:
        state[4, 1] = 7
    parents = rng.integers(-1, R, R).astype(np.int32)
    recent = rng.integers(0, 1 << 16, (2 * R + 3, H, 2, 64 * D)).astype(np.uint16)
    dev = up(recent.view(np.int16)).view(torch.bfloat16)
    for _ in range(2):                                                     # the second time writes the same
        jf.kv_fork_recent(up(parents), up(state), dev)
    ro.fork_recent(parents, state, recent)
    assert np.array_equal(dev.view(torch.int16).cpu().numpy().view(np.uint16), recent)


# ------------------------------------------------------------------------------------------------ sweep
def cache_state(rng, R, width, blocks, share):
    state = np.stack([rng.integers(0, 64 * width + 64, R), rng.integers(0, 2, R)], 1).astype(np.int32)
    state[rng.random(R) < 0.3, 0] = 0
    table = rng.integers(0, max(1, int(blocks * share)), (R, width)).astype(np.int32)
    odd = rng.random((R, width)) < 0.02
    table[odd] = rng.choice([-1, -5, blocks, blocks + 9, 2 ** 31 - 1], odd.sum())
    return state, table


@pytest.mark.parametrize("share", [0.01, 0.6, 1.0])
@pytest.mark.parametrize("R,width,blocks", [(1, 1, 1), (1, 3, 2), (3, 8, 63), (10, 5, 64), (20, 30, 65), (64, 128, 4000), (65, 128, 4096),
                                            (300, 200, 20000), (4096, 130, 100000), (50, 40, 1 << 18)])
def test_sweep(jf, R, width, blocks, share):
    rng = np.random.default_rng(R + blocks)
    state, table = cache_state(rng, R, width, blocks, share)
    for compact in (False, True):
        got = jf.kv_sweep(up(state), up(table), blocks, compact=compact)
        want = ro.sweep(state, table, blocks, compact)
        for k, v in want.items():
            g = getattr(got, k)
            assert (g is None) == (v is None), k
            if v is not None:
                assert np.array_equal(g.cpu().numpy(), v), k


def test_sweep_full_and_empty(jf):
    """Nobody holds anything; every block is held; one block is left."""
    for blocks in (64, 100, 129):
        table = np.arange(blocks, dtype=np.int32)[::-1][None].copy()
        for held in (0, blocks - 1, blocks):
            state = np.array([[64 * held + 3, 0]], np.int32)
            for compact in (False, True):
                got, want = jf.kv_sweep(up(state), up(table), blocks, compact=compact), ro.sweep(state, table, blocks, compact)
                for k, v in want.items():
                    assert v is None or np.array_equal(getattr(got, k).cpu().numpy(), v), (blocks, held, k)


@pytest.mark.parametrize("H,D", [(1, 64), (3, 128), (8, 128)])
def test_moves(jf, H, D):
    """A compaction's moves, with ids that are none of the cache between them: every table reads the same blocks as before."""
    import torch
    rng = np.random.default_rng(D)
    R, width, blocks = 12, 20, 300
    state, table = cache_state(rng, R, width, blocks, 1.0)
    codes = rng.integers(0, 256, (blocks, H, 2, 64 * D)).astype(np.uint8)
    scales = rng.random((blocks, H, 2), dtype=np.float32)
    p = jf.kv_sweep(up(state), up(table), blocks, compact=True)
    c, s = up(codes), up(scales)
    moves = torch.cat([p.moves, torch.tensor([[-1, 3], [3, -1], [blocks, 2], [2, blocks + 7], [5, 5]], dtype=torch.int32).cuda()])
    for _ in range(2):
        jf.kv_move(moves, c, s)
    new, live = p.next_table.cpu().numpy(), int(p.live)
    c, s = c.cpu().numpy(), s.cpu().numpy()
    for r in range(R):
        for j in range(min(state[r, 0] // 64, width)):
            old = table[r, j]
            if not 0 <= old < blocks:
                assert new[r, j] == -1
                continue
            assert 0 <= new[r, j] < live
            assert np.array_equal(c[new[r, j]], codes[old]) and np.array_equal(s[new[r, j]], scales[old])
        assert (new[r, min(state[r, 0] // 64, width):] == -1).all()
    untouched = [b for b in range(blocks) if b not in set(p.moves.cpu().numpy()[:, 1].tolist())]
    assert np.array_equal(c[untouched], codes[untouched])


def test_moves_of_large_caches(jf):
    """Offsets behind 2^32 bytes."""
    import torch
    blocks, H, D = 40000, 8, 128                                           # 5.2 GB of codes
    codes = torch.zeros((blocks, H, 2, 64 * D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((blocks, H, 2), device="cuda")
    codes[-1] = torch.randint(0, 256, codes[-1].shape, dtype=torch.uint8, device="cuda")
    scales[-1] = 3.0
    jf.kv_move(torch.tensor([[blocks - 1, 36000], [36001, 1]], dtype=torch.int32, device="cuda"), codes, scales)
    assert torch.equal(codes[36000], codes[-1]) and (scales[36000] == 3).all()
    assert not codes[1].any() and not codes[35999].any() and not codes[36001].any()


# ------------------------------------------------------------------------------------------------ use
def test_swept_blocks_are_planned_again(jf):
    """Ends, forks, sweep and plan in turn: no block is handed out while somebody holds it, and none is lost."""
    rng = np.random.default_rng(0)
    R, width, blocks = 30, 12, 200
    state, table = np.zeros((R, 2), np.int32), np.full((R, width), -1, np.int32)
    dstate, dtable = up(state), up(table)
    sweep = jf.kv_sweep(dstate, dtable, blocks)
    for step in range(25):
        lens = rng.integers(0, 90, R)
        lens = np.where(state[:, 0] + lens > 64 * width, 0, lens).astype(np.int32)
        p = jf.kv_plan(dstate, up(lens), sweep.free_blocks, sweep.free_head, dtable, max(1, int(lens.sum())), 90)
        state = p.next_state.cpu().numpy()
        held = [set(row[:n // 64].tolist()) for row, n in zip(dtable.cpu().numpy(), state[:, 0])]
        assert all(0 <= b < blocks for h in held for b in h) and all(len(h) == n // 64 for h, n in zip(held, state[:, 0]))
        over = rng.random(R) < 0.3
        state = np.where(over[:, None], [0, 0], state).astype(np.int32)
        parents = np.where(rng.random(R) < 0.3, rng.integers(0, R, R), -1).astype(np.int32)
        f = jf.kv_fork(up(state), dtable, up(parents))
        dstate, dtable, state = f.next_state, f.next_table, f.next_state.cpu().numpy()
        sweep = jf.kv_sweep(dstate, dtable, blocks, compact=step % 3 == 0)
        if step % 3 == 0:
            dtable = sweep.next_table
        live = {b for row, n in zip(dtable.cpu().numpy(), state[:, 0]) for b in row[:n // 64].tolist()}
        free = sweep.free_blocks.cpu().numpy()
        free = set(free[free >= 0].tolist())
        assert not live & free and live | free == set(range(blocks)) and int(sweep.live) == len(live)


def test_streams_and_graphs(jf):
    import torch
    rng = np.random.default_rng(2)
    R, width, blocks = 200, 100, 3000
    state, table = cache_state(rng, R, width, blocks, 0.7)
    s, t, parents = up(state), up(table), up(rng.integers(-1, R, R).astype(np.int32))
    want, fork = jf.kv_sweep(s, t, blocks, compact=True), jf.kv_fork(s, t, parents)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [jf.kv_sweep(s, t, blocks, compact=True, stream=x) + jf.kv_fork(s, t, parents, stream=x) for x in streams]
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(want + fork, out))
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(jf.kv_sweep_workspace(R, width, blocks), dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        captured = jf.kv_sweep(s, t, blocks, compact=True, workspace=ws) + jf.kv_fork(s, t, parents)
    for n in range(3):
        state, table = cache_state(rng, R, width, blocks, 0.2 + 0.3 * n)
        s.copy_(up(state))
        t.copy_(up(table))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(jf.kv_sweep(s, t, blocks, compact=True) + jf.kv_fork(s, t, parents), captured):
            assert torch.equal(a, b)


def test_binding_refusals(jf):
    import torch
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    for f in (lambda: jf.kv_positions(i(4, 7), 4), lambda: jf.kv_prefix(i(4, 8), i(3, 8), i(2)),
              lambda: jf.kv_fork(i(3, 2), i(2, 8), i(3)), lambda: jf.kv_fork(i(2, 2), i(2, 8), i(3)),
              lambda: jf.kv_sweep(i(3, 2), i(2, 8), 10),
              lambda: jf.kv_fork_recent(i(2), i(3, 2), torch.zeros((6, 1, 2, 64 * 64), dtype=torch.bfloat16, device="cuda")),
              lambda: jf.kv_move(i(4, 3), torch.zeros((4, 1, 2, 64 * 64), dtype=torch.uint8, device="cuda"),
                                 torch.zeros((4, 1, 2), device="cuda"))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        jf.kv_fork(i(2, 2), i(2, 8), i(2).long())
    with pytest.raises(jf.JetFP8Error):
        jf.kv_sweep(i(2, 2), i(2, 8), (1 << 18) + 1)
    with pytest.raises(jf.JetFP8Error):
        jf.kv_fork_recent(i(4), i(4, 2), torch.zeros((7, 1, 2, 64 * 64), dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("R,W", [(8, 16), (70, 128)])
def test_tables_side_by_side(jf, R, W):
    """The tables before and after may be neighbours in one buffer; in place they are refused and nothing is written."""
    import torch
    rng = np.random.default_rng(4)
    state = np.stack([rng.integers(0, 64 * W, R), rng.integers(0, 2, R)], 1).astype(np.int32)
    table = rng.integers(0, 300, (R, W)).astype(np.int32)
    parents = rng.integers(-1, R, R).astype(np.int32)
    both, states = torch.zeros((2, R, W), dtype=torch.int32, device="cuda"), torch.zeros((2, R, 2), dtype=torch.int32, device="cuda")
    both[0], states[0] = up(table), up(state)
    new = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    free, head, live, moves = new(300), new(1), new(1), new(150, 2)
    ws = torch.empty(max(16, jf.kv_sweep_workspace(R, W, 300)), dtype=torch.uint8, device="cuda")
    jf.jetfp8_kv_fork(states[0], both[0], W, R, up(parents), states[1], both[1])
    s, t = ro.fork(state, table, parents)
    assert np.array_equal(states[1].cpu().numpy(), s) and np.array_equal(both[1].cpu().numpy(), t)
    jf.jetfp8_kv_sweep(states[0], both[0], W, R, 300, free, head, live, both[1], moves, ws)
    assert np.array_equal(both[1].cpu().numpy(), ro.sweep(state, table, 300, True)["next_table"])
    for f in (lambda: jf.jetfp8_kv_fork(states[0], both[0], W, R, up(parents), states[0], both[1]),
              lambda: jf.jetfp8_kv_fork(states[0], both[0], W, R, up(parents), states[1], both[0]),
              lambda: jf.jetfp8_kv_sweep(states[0], both[0], W, R, 300, free, head, live, both[0], moves, ws)):
        with pytest.raises(jf.JetFP8Error):
            f()
    assert np.array_equal(both[0].cpu().numpy(), table) and np.array_equal(states[0].cpu().numpy(), state)
