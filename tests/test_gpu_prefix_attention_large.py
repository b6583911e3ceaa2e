"""The tests of shared prompts once more with bounds so large (the call may read 1 GiB) that every form with up to 32 rows a
unit takes the shared blocks apart, and which calls do at all."""
import numpy as np
import pytest

import test_gpu_prefix_attention as base
from test_gpu_prefix_attention import (Case, jf, same, test_against_the_oracle, test_bits_of_the_plain_attention, test_codes,  # noqa: F401
                                       test_ids_of_no_block_and_zero_scales, test_records_of_other_units, test_rows_of_many_parts,
                                       test_several_tokens_and_idle_requests, test_streams_and_graphs, test_values_of_every_size)

pytestmark = pytest.mark.gpu


def reads(c, size):
    """A max_seq with which the call may read `size` bytes."""
    return max(c.max_seq, 64 * max(256, -(-size // (len(c.units) * c.H * 128 * c.D))) + 1)


@pytest.fixture(autouse=True)
def far(monkeypatch):
    monkeypatch.setattr(base.Case, "far", lambda c: reads(c, 1 << 30))


def apart(jf, c, max_seq):
    """Whether a call takes shared blocks apart: the first unit's first span then has no partial result of its own."""
    import torch
    pre = c.prefix(jf)
    assert int(pre[0, 2]) >= 16
    need = jf.attention_workspace(len(c.units), c.new, max_seq, c.Hq, c.H, c.D, True)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    jf.attention(c.q, *c.args(), max_new=c.new, max_seq=max_seq, prefix=pre, workspace=ws)
    return bool((ws[:4 * c.D] == 255).all()) if need else False


@pytest.mark.parametrize("Hq,H,D,new,prompt,samples,mib,yes", [
    (4, 1, 128, 1, 1100, 4, 512, True), (16, 1, 128, 1, 1100, 4, 256, True), (32, 1, 128, 1, 1100, 4, 1024, True),
    (32, 1, 128, 1, 1100, 4, 512, False), (33, 1, 128, 1, 1100, 4, 1024, False),
    (8, 1, 64, 1, 1100, 4, 256, True), (8, 1, 64, 1, 1100, 4, 255, False),
    (32, 8, 128, 1, 1500, 24, 384, True), (32, 8, 128, 1, 1500, 24, 383, False), (32, 8, 64, 1, 1500, 24, 383, True),
    (8, 8, 64, 1, 1471, 200, 0, False), (8, 8, 64, 1, 1537, 200, 0, True),
    (64, 8, 128, 4, 1600, 70, 0, True), (64, 8, 64, 4, 3000, 70, 0, False), (64, 8, 64, 4, 3100, 70, 0, True)])
def test_which_calls(jf, Hq, H, D, new, prompt, samples, mib, yes):
    """By rows, blocks, and what the call may read: 256 MiB (64 channels, or 256 blocks and more) or 384, of 24 blocks a request
    and more; above 16 rows 1 GiB, or 1024 waves of 24 blocks (64 channels: 48).  The results are the same."""
    c = Case([(prompt, samples)], 0, new, Hq, H, D, seed=1)
    per = len(c.units) * H * 128 * D
    max_seq = max(c.max_seq, 64 * (-(-(mib << 20) // per) if yes else ((mib << 20) + (1 << 19)) // per) + 1)
    assert apart(jf, c, max_seq) == yes
    same(c.run(jf, c.prefix(jf), max_seq), c.run(jf, None, c.max_seq))


def test_a_part_of_the_units(jf):
    """Records of single units make the plain call of any part of a plan's."""
    import torch
    c = Case([(1100, 8), (600, 3)], 100, 1, 4, 2, 128, seed=2)
    plain = c.run(jf, None, c.max_seq)
    u = c.units[3:9].contiguous()
    alone = torch.tensor([[i, 1, 0, 0] for i in range(6)], dtype=torch.int32, device="cuda")
    o = torch.full_like(plain, 7.0)
    top = 64 * ((1 << 30) // (6 * 2 * 128 * 128)) + 65
    ws = torch.empty(jf.attention_workspace(6, 1, top, 4, 2, 128, True), dtype=torch.uint8, device="cuda")
    jf.jetfp8_attention_prefix(c.q, u, alone, c.table, c.dcodes, c.dscales, c.recent, c.T, 1, top, 4, 2, 128, 128 ** -0.5, o,
                               workspace=ws)
    same(o[3:9], plain[3:9])
    assert (o[:3] == 7.0).all() and (o[9:] == 7.0).all()


@pytest.mark.parametrize("Hq,H,D,new,idle", [(3, 1, 64, 1, 0.0), (16, 2, 64, 1, 0.1), (5, 1, 128, 2, 0.3)])
def test_more_units_than_threads(jf, Hq, H, D, new, idle):
    """1500 requests: each thread that counts pieces has several units, and groups begin and end within a thread's."""
    c = Case([(520, 700), (1100, 499), (100, 2), (2100, 300)], 100, new, Hq, H, D, idle=idle, seed=Hq)
    assert len(c.units) > 1024
    pre = c.prefix(jf)
    same(c.run(jf, pre, c.far()), c.run(jf, None, c.max_seq))
