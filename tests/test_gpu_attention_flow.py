"""A stack of FP8 pre-norm decoder blocks that runs on the library's kernels alone: norm, QKV, the key/value cache and its
attention with fused codes, output projection, norm, gate/up, SwiGLU, down projection (Jet-RL explainers, "Architecture
Centrale": the rollout graph is a subgraph of the training forward graph, with the same quantization and precision).
Every hidden state of a token is bitwise the same in a prompt of the whole sequence, in single-token decoding beside
other requests, and in chunks of any size; and the attention differs from that over bf16 keys and values by the cache's
quantization error.  Weights are random and seeded; no trained model is involved."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

DM, HQ, HKV, HD, F, LAYERS, S = 1024, 8, 2, 128, 2816, 3, 300
QKV = (HQ + 2 * HKV) * HD
EPS = 1e-5


@pytest.fixture(scope="module")
def stack():
    import torch
    import fp8_precision_rl_amd as jf
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    jf.load_library()
    g = torch.Generator(device="cuda")
    g.manual_seed(11)

    def lin(n, k):
        return jf.quantize_blocks((torch.randn((n, k), device="cuda", generator=g) * k ** -0.5).to(torch.bfloat16), False)

    norm = lambda: (1.0 + 0.1 * torch.randn((DM,), device="cuda", generator=g)).to(torch.bfloat16)
    layers = [dict(qkv=lin(QKV, DM), o=lin(DM, HQ * HD), gu=lin(2 * F, DM), dn=lin(DM, F), n1=norm(), n2=norm())
              for _ in range(LAYERS)]
    x0 = torch.randn((S, DM), device="cuda", generator=g).to(torch.bfloat16)
    x0[:, 17] *= 30                                                   # an outlier channel
    return jf, layers, x0


class Rollout:
    """R requests fed the same sequence, `others` tokens of it behind one another's."""

    def __init__(self, jf, layers, R, tokens):
        import torch
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
        self.jf, self.layers, self.R = jf, layers, R
        width = S // 64 + 1
        self.caches = [jf.kv_cache(R * width, R, tokens, HKV, HD) for _ in layers]
        self.state, self.head = torch.zeros((R, 2), dtype=torch.int32, device="cuda"), i32(0)
        self.free = torch.randperm(R * width, device="cuda").to(torch.int32)
        self.table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")

    def step(self, x, lens):
        """x: the step's rows, request by request; returns the hidden states after every block."""
        import torch
        jf = self.jf
        T, n = len(x), torch.tensor(lens, dtype=torch.int32, device="cuda")
        p = jf.kv_plan(self.state, n, self.free, self.head, self.table, T, max(lens))
        outs = []
        for L, cache in zip(self.layers, self.caches):
            xq, xs, _ = jf.rmsnorm_quantize(x, L["n1"], EPS)
            qkv = jf.gemm_fwd(xq, xs, *L["qkv"]).view(T, HQ + 2 * HKV, HD)
            jf.kv_append(qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], p.units, *cache)
            aq, as_ = jf.attention(qkv[:, :HQ], p.units, self.table, *cache, max_new=max(lens), max_seq=S, quantize=True,
                                   return_o=False)
            h = (x.float() + jf.gemm_fwd(aq, as_, *L["o"]).float()).to(torch.bfloat16)
            hq, hs, _ = jf.rmsnorm_quantize(h, L["n2"], EPS)
            sq, ss = jf.swiglu_quantize(jf.gemm_fwd(hq, hs, *L["gu"]))
            x = (h.float() + jf.gemm_fwd(sq, ss, *L["dn"]).float()).to(torch.bfloat16)
            outs.append(x)
        self.state, self.head = p.next_state, p.next_free
        assert not p.status.any()
        return outs


@pytest.mark.parametrize("cut", ["tokens", "halves", "ragged", "batch"])
def test_hidden_states_do_not_depend_on_the_cut(stack, cut):
    import torch
    jf, layers, x0 = stack
    whole = Rollout(jf, layers, 1, S).step(x0, [S])
    if cut == "batch":            # many prompts at once: the serial attention kernel
        R = 40
        run = Rollout(jf, layers, R, R * S)
        outs = [o[7 * S:8 * S] for o in run.step(x0.repeat(R, 1), [S] * R)]
    else:
        sizes = {"tokens": [1] * S, "halves": [150, 150], "ragged": [70, 1, 63, 2, 128, 36]}[cut]
        R = 3
        run = Rollout(jf, layers, R, R * max(sizes))
        outs, at = [[] for _ in layers], 0
        for n in sizes:
            x = torch.cat([x0[at:at + n].flip(0), x0[at:at + n], x0[at:at + n] * 0.5])
            for have, o in zip(outs, run.step(x, [n] * R)):
                have.append(o[n:2 * n])
            at += n
        outs = [torch.cat(o) for o in outs]
    for depth, (a, b) in enumerate(zip(whole, outs)):
        diff = (a.view(torch.int16) != b.view(torch.int16)).any(dim=1).nonzero().flatten()
        assert len(diff) == 0, f"{cut}: tokens {diff[:8].tolist()} differ at depth {depth}"


def test_attention_error_of_the_cache(stack):
    """The FP8 cache against float64 attention over the bf16 keys and values.  E4M3 rounds a normal code by at most 2^-4
    of it, so each score moves by at most 2^-4 sum |q k| and each value by 2^-4 of itself; for random data the
    relative error of the result stays below that of one code."""
    import torch
    jf, _, _ = stack
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    qkv = torch.randn((S, HQ + 2 * HKV, HD), device="cuda", generator=g).to(torch.bfloat16)
    run = Rollout(jf, [None], 1, S)
    p = jf.kv_plan(run.state, torch.tensor([S], dtype=torch.int32, device="cuda"), run.free, run.head, run.table, S, S)
    jf.kv_append(qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], p.units, *run.caches[0])
    o = jf.attention(qkv[:, :HQ], p.units, run.table, *run.caches[0], max_new=S, max_seq=S).double().cpu().numpy()
    q, k, v = (t.double().cpu().numpy() for t in (qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]))
    k, v = (np.repeat(t, HQ // HKV, 1) for t in (k, v))
    s = np.einsum("thd,nhd->htn", q, k) * HD ** -0.5
    s = np.where(np.tril(np.ones((S, S), bool)), s, -np.inf)
    e = np.exp(s - s.max(-1, keepdims=True))
    want = np.einsum("htn,nhd->thd", e / e.sum(-1, keepdims=True), v)
    rel = np.linalg.norm(o - want) / np.linalg.norm(want)
    first = np.linalg.norm(o[:64] - want[:64]) / np.linalg.norm(want[:64])
    print(f"relative error {rel:.3e}; tokens of the first block, which read no codes, {first:.3e}", flush=True)
    assert rel < 2.0 ** -4 and first < 2.0 ** -8
