"""An attention layer from projection to projection: gdn_quant_linear,
gdn_kv_write_m with its rotation, gdn_attn_step_m, gdn_quant_linear; prompts by
chunks, single tokens, drafted tokens and their rollback, captured steps."""

import pytest
import torch

import gated_deltanet_linear_gb300 as gdn
from attn_ref import KINDS, codes, turn
from linattn_ref import make_quant, quant_linear

pytestmark = pytest.mark.gpu

QH, KVH, HD, ROT, PAGE, K = 6, 2, 64, 32, 16, 256
N = (QH + 2 * KVH) * HD


class Layer:
    """B sequences with pages of their own, and the 64-bit form beside."""

    def __init__(self, kind, dtype, B=3, cols=12, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kind, self.dtype, self.B, self.gen = kind, dtype, B, g
        self.w_in, self.w_out = (self._weights(g, n, k) for n, k in ((N, K), (K, QH * HD)))
        f, _ = gdn.gdn_rope_freqs(ROT, 1e5)
        self.freq, self.rope = f, gdn.Rope(f)
        pages = B * cols
        k = torch.zeros(pages, KVH, PAGE, HD, device="cuda").to(KINDS[kind])
        s = None if kind == "bf16" else torch.zeros(pages, KVH, PAGE, device="cuda")
        self.cache = gdn.KVCache(k, k.clone(), s, None if s is None else s.clone())
        self.table = torch.randperm(pages, generator=g, device="cuda").int().view(B, cols)
        self.start = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(gdn.gdn_attn_workspace(self.cache, 8, QH), dtype=torch.uint8, device="cuda")
        self.hist = [(torch.zeros(0, KVH, HD, dtype=torch.float64, device="cuda"),) * 2 for _ in range(B)]

    @staticmethod
    def _weights(g, n, k):
        qw = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        sc = (torch.exp(0.2 * torch.randn(n, k // 64, generator=g, device="cuda")) / (4.0 * k ** 0.5)).half()
        return qw, sc

    def tokens(self, M):
        return torch.randn(self.B, M, K, generator=self.gen, device="cuda").to(self.dtype)

    def write(self, x):
        """The projection and the cache's rows; returns q."""
        B, M, _ = x.shape
        p = torch.empty(B * M, N, device="cuda", dtype=self.dtype)
        gdn.gdn_quant_linear(x.view(B * M, K), *self.w_in, p)
        p = p.view(B, M, QH + 2 * KVH, HD)
        q = torch.empty(B, M, QH, HD, device="cuda", dtype=self.dtype)
        gdn.gdn_kv_write_m(self.cache, p[:, :, QH:QH + KVH], p[:, :, QH + KVH:], self.table, self.start,
                           rope=self.rope, q=p[:, :, :QH], q_out=q)
        return p, q

    def step(self, x):
        B, M, _ = x.shape
        p, q = self.write(x)
        o = torch.empty_like(q)
        gdn.gdn_attn_step_m(self.cache, q, self.table, self.start, o, workspace=self.ws)
        y = torch.empty(B * M, K, device="cuda", dtype=self.dtype)
        gdn.gdn_quant_linear(o.view(B * M, QH * HD), *self.w_out, y)
        return p, o, y.view(B, M, K)

    def held(self, x):
        if self.kind == "bf16":
            return x.float().bfloat16().double()
        c, s = codes(x, self.kind)
        return c * s.double()[..., None]

    def expect(self, p, keep):
        """o in 64 bits from the projection's own output p; the first `keep`
        tokens stay in the history."""
        B, M = p.shape[:2]
        out = torch.zeros(B, M, QH, HD, dtype=torch.float64, device="cuda")
        for b in range(B):
            pos = int(self.start[b]) + torch.arange(M, device="cuda")
            q = turn(p[b, :, :QH], pos, self.freq, False, 1.0)
            k = self.held(turn(p[b, :, QH:QH + KVH], pos, self.freq, False, 1.0))
            v = self.held(p[b, :, QH + KVH:].double())
            hk, hv = (torch.cat([h, n]) for h, n in zip(self.hist[b], (k, v)))
            for m in range(M):
                n = int(self.start[b]) + m + 1
                x = q[m].view(KVH, QH // KVH, HD)
                w = torch.softmax(torch.einsum("hgd,thd->hgt", x, hk[:n]) * HD ** -0.5, -1)
                out[b, m] = torch.einsum("hgt,thd->hgd", w, hv[:n]).reshape(QH, HD)
            n = int(self.start[b]) + keep
            self.hist[b] = (hk[:n], hv[:n])
        return out


def near(o, want, kind, dtype):
    """Codes of turned keys may lie one step off where the turn's rounding meets a
    border (one element in 10^4): a score is then off by a code of one channel,
    |q| amax / 127 (e4m3: a sixteenth of the element) over HD ^ 0.5, some
    hundredths, for one key; on 40 and more keys 1e-3 of o's size covers it
    beside the type's rounding (bf16 2^-8, and as much for its q)."""
    tol = (2.0 ** -7 if dtype == torch.bfloat16 else 0.0) + (2e-3 if kind != "e4m3" else 6e-3)
    return ((o.double() - want).norm() / want.norm()).item() <= tol


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_steps_and_rollback(kind, dtype):
    L = Layer(kind, dtype)
    for M in (8, 8, 8, 5, 8, 8):                    # a prompt by chunks
        p, o, y = L.step(L.tokens(M))
        want = L.expect(p, M)
        assert near(o, want, kind, dtype)
        ref = quant_linear(o.reshape(-1, QH * HD), *L.w_out)[0]
        tol = 2.0 ** -8 if dtype == torch.bfloat16 else 1e-5
        assert (y.reshape(-1, K).double() - ref).norm() <= tol * ref.norm()
        L.start += M
    for _ in range(4):                               # single tokens
        p, o, _ = L.step(L.tokens(1))
        assert near(o, L.expect(p, 1), kind, dtype)
        L.start += 1
    # four drafted tokens at once are the four one by one
    x = L.tokens(4)
    start = L.start.clone()
    p4, o4, _ = L.step(x)
    for m in range(4):
        p, o, _ = L.step(x[:, m:m + 1].contiguous())
        assert (o[:, 0].double() - o4[:, m].double()).norm() <= (2e-5 if dtype == torch.float32 else 2.0 ** -7) * o4[:, m].double().norm()
        L.start += 1
    # two of them accepted: the cursor goes back and the next token is written
    # over the third
    L.start.copy_(start)
    L.expect(p4, 2)
    L.start += 2
    p, o, _ = L.step(L.tokens(1))
    assert near(o, L.expect(p, 1), kind, dtype)


def test_captured_layer_runs_on():
    """A captured step with the cursor moved inside the graph, replayed over
    page ends, is the same as eager steps."""
    A, B = Layer("int8", torch.bfloat16, seed=1), Layer("int8", torch.bfloat16, seed=1)
    x = torch.zeros(A.B, 1, K, device="cuda", dtype=torch.bfloat16)
    g = torch.cuda.CUDAGraph()
    A.step(x)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        _, oa, ya = A.step(x)
        A.start += 1
    A.start.zero_()
    for _ in range(40):
        t = torch.randn(x.shape, generator=A.gen, device="cuda").to(x.dtype)
        x.copy_(t)
        g.replay()
        _, ob, yb = B.step(t)
        B.start += 1
        assert torch.equal(oa, ob) and torch.equal(ya, yb)
    assert torch.equal(A.cache.k, B.cache.k) and torch.equal(A.cache.v_scale, B.cache.v_scale)
    assert int(A.start[0]) == 40 and gdn.gdn_wait_timeouts() == 0


def test_two_graphs_share_a_workspace():
    """Two captured steps of different batches, one workspace, replayed in turn
    on one stream."""
    A, B = Layer("e4m3", torch.float32, B=2, seed=2), Layer("bf16", torch.float32, B=5, seed=3)
    ws = A.ws if A.ws.numel() >= B.ws.numel() else B.ws
    A.ws = B.ws = ws
    runs = []
    for L in (A, B):
        for M in (8, 8, 8, 8, 8):
            L.write(L.tokens(M))
            L.start += M
        x = L.tokens(2)
        _, want, _ = L.step(x)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _, o, _ = L.step(x)
        runs.append((g, o, want.clone(), x))  # (x is read by every replay)
    for _ in range(3):
        for g, *_ in runs:
            g.replay()
        for _, o, want, _ in runs:
            assert torch.equal(o, want)


def test_shared_prefix_pages():
    """Two sequences whose tables name the same pages for their first tokens."""
    L = Layer("int8", torch.float32, B=2, seed=4)
    L.table[1, :3] = L.table[0, :3]
    x = L.tokens(48)
    x[1] = x[0]
    both = L.table.clone()
    L.table[1, :3] = L.table[1, 6:9]           # the prompt is written once
    L.write(x)
    L.table.copy_(both)
    L.start += 48
    x = L.tokens(1)
    x[1] = x[0]
    _, o, _ = L.step(x)
    assert torch.equal(o[0], o[1])
    x = L.tokens(1)                             # and then they part
    L.start += 1
    _, o, _ = L.step(x)
    assert not torch.equal(o[0], o[1])
