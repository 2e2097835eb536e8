"""New tokens chained with the sparse attention on one stream: norm, append, prefix attention and
the sparse calls in CUDA graphs, where nothing but the kernels' own waits keeps them apart.

Every graph is replayed on changed inputs, with its intermediate queries filled with other numbers
beforehand, and has to give the bits of the same calls with a synchronise after each.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def skv():
    import __graft_entry__

    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


class Layer:
    """A paged pool of `B` requests, a batch of new tokens -- chunks of their prompts and, last, the
    token that ends each history -- and a fixed selection of the histories."""

    def __init__(self, skv, B, H, G, L, k, chunk, dtype, prefix=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.skv, self.B, self.H, self.G, self.g, self.dtype = skv, B, H, G, g, dtype
        bs, cap = 16, L + 16
        per = (cap + bs - 1) // bs
        self.pk, self.pv = (torch.randn((B * per, H, bs, D), generator=g).to(dtype).cuda() for _ in range(2))
        table = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per)
        if prefix:
            table[:, :prefix // bs] = table[0, :prefix // bs].clone()
        self.lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
        self.p = skv.Problem(batch=B, n_kv_heads=H, n_q_heads=H * G, d_qk=D, d_v=D, max_len=cap, topk=k, n_sink=0,
                             n_local=16, block_size=bs, seq_lens=self.lens,
                             dtype=skv.SKV_DTYPE_F32 if dtype == torch.float32 else skv.SKV_DTYPE_BF16)
        self.pool = skv.Pool(self.pk, self.pv, table.cuda())
        self.prefix = skv.Prefix(table[0, :(prefix + bs - 1) // bs].contiguous().cuda(), prefix) if prefix else None
        self.n = chunk + B
        share = max((chunk + B - 1) // B, 1)
        assert share < L
        i = torch.arange(chunk, dtype=torch.int32)
        self.pos = torch.cat([i % share, torch.full((B,), L - 1, dtype=torch.int32)]).cuda()
        self.req = torch.cat([i // share, torch.arange(B, dtype=torch.int32)]).cuda()
        # the norm alone turns every row
        self.every = torch.randint(0, L, (self.n,), generator=g).to(torch.int32).cuda()
        inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        gam = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2)]
        self.tokens = skv.TokenStep(self.p, skv.Rotary(inv.float().cuda(), rot_dim=D, q_gamma=gam[0], k_gamma=gam[1]),
                                    self.pool)
        self.q, self.k, self.v = (torch.empty((self.n, h, D), dtype=dtype, device="cuda") for h in (H * G, H, H))
        self.q_out, self.k_out = torch.empty_like(self.q), torch.empty_like(self.k)
        idx = torch.stack([torch.randperm(L - 16, generator=g)[:k].sort().values for _ in range(B * H)])
        self.idx = idx.to(torch.int32).view(B, H, k).cuda()
        self.out = torch.empty((B, H * G, D), dtype=dtype, device="cuda")
        self.lse = torch.empty((B, H * G), device="cuda")
        self.ws = torch.empty(max(skv.skv_workspace_size(self.p), 16), dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def fresh(self):
        for t in (self.q, self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=self.g).to(self.dtype))
        for t in (self.q_out, self.k_out, self.out, self.lse):
            t.fill_(5.0)
        torch.cuda.synchronize()

    @property
    def mine(self):
        """The decode tokens' queries, written last."""
        return self.q_out[self.n - self.B:]

    def append(self):
        self.tokens.append(self.q, self.k, self.v, self.pos, self.req, q_out=self.q_out)

    def norm(self):
        self.tokens.norm_rope(self.q, self.k, self.every, q_out=self.q_out, k_out=self.k_out)

    def sparse(self):
        self.skv.skv_sparse_attn(self.p, self.mine, self.pool, self.idx, self.out, self.lse, self.ws, self.status)


def _replays(layer, calls, results, times=6):
    """calls in one graph against calls synchronised one by one."""
    layer.fresh()
    for c in calls:  # (kernels' attributes are set before the capture)
        c()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    pools = [layer.pk.clone(), layer.pv.clone()]
    for _ in range(times):
        layer.fresh()
        layer.pk.copy_(pools[0]), layer.pv.copy_(pools[1])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in results()]
        for t in (layer.q_out, layer.k_out, layer.out, layer.lse):
            t.fill_(7.0)
        layer.pk.copy_(pools[0]), layer.pv.copy_(pools[1])
        torch.cuda.synchronize()
        for c in calls:
            c()
            torch.cuda.synchronize()
        for a, b in zip(got, results()):
            assert torch.equal(a, b)
    assert int(layer.status.item()) == 0 and int(layer.tokens.status.item()) == 0


SHAPES = [
    # B, H, G, L, k, chunk tokens, dtype
    (8, 8, 8, 2048, 300, 4000, torch.bfloat16),   # splits merged in a cluster
    (1, 1, 8, 4096, 3000, 3900, torch.bfloat16),  # and through the workspace
    (3, 2, 16, 700, 64, 2000, torch.bfloat16),    # heads on the other side of the product
    (4, 2, 4, 700, 64, 0, torch.bfloat16),        # one token a request alone
    (2, 2, 4, 700, 64, 1300, torch.float32),
]


@pytest.mark.parametrize("shape", SHAPES)
def test_append_then_sparse_attention(skv, shape):
    x = Layer(skv, *shape, seed=1)
    _replays(x, [x.append, x.sparse], lambda: (x.mine, x.out, x.lse, x.pk, x.pv))


@pytest.mark.parametrize("shape", SHAPES)
def test_norm_then_sparse_attention(skv, shape):
    x = Layer(skv, *shape, seed=2)
    _replays(x, [x.norm, x.sparse], lambda: (x.mine, x.out, x.lse))


@pytest.mark.parametrize("shape", SHAPES[:4])
def test_norm_then_prefix_then_sparse_attention(skv, shape):
    """The prefix attention's kernels release their successors as they start, too."""
    x = Layer(skv, *shape, seed=3, prefix=320)
    step = skv.PrefixStep(x.p, x.pool, x.prefix)
    x.fresh()
    _replays(x, [x.norm, lambda: step.run(x.mine), x.sparse], lambda: (x.mine, step.out, step.lse, x.out, x.lse))
    assert int(step.status.item()) == 0


@pytest.mark.parametrize("shape", SHAPES)
def test_append_then_decode_step(skv, shape):
    """The whole step on the appended pool: it scores, selects and attends what was just written."""
    x = Layer(skv, *shape, seed=4)
    step = skv.DecodeStep(x.p, x.pool, x.mine, skv.IndexSrc())
    _replays(x, [x.append, step.run], lambda: (x.mine, step.idx, step.out, step.lse))
    assert int(step.status.item()) == 0


def test_lengths_counted_in_the_graph(skv):
    """A decode loop's graph: the lengths advance, the token is appended at the new end and attended."""
    x = Layer(skv, 4, 2, 8, 512, 40, 0, torch.bfloat16, seed=5)

    def token():
        x.tokens.append(x.q, x.k, x.v, q_out=x.q_out)

    calls = [lambda: x.lens.add_(1), token, x.sparse]
    x.fresh()
    for c in calls:
        c()
    torch.cuda.synchronize()
    x.lens.fill_(512)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    for it in range(8):
        x.fresh()
        before = [x.pk.clone(), x.pv.clone(), x.lens.clone()]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (x.q_out, x.out, x.lse, x.pk, x.pv, x.lens)]
        x.pk.copy_(before[0]), x.pv.copy_(before[1]), x.lens.copy_(before[2])
        for c in calls:
            c()
            torch.cuda.synchronize()
        for a, b in zip(got, (x.q_out, x.out, x.lse, x.pk, x.pv, x.lens)):
            assert torch.equal(a, b)
    assert int(x.status.item()) == 0 and int(x.tokens.status.item()) == 0
