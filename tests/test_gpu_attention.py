"""Attention with a bucketed relative bias on the GPU, forward and backward, against the 64-bit
reference (block_reference.py holds it and the derivation of the bounds)."""
import math

import pytest
import torch

import block_reference as ref
from block_reference import DT
from spatial_transformer_sampling_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "float16", "bfloat16"]


def _draw(g, shape, dtype, std=1.0):
    return wl.as_dtype(g.normal(size=shape) * std, dtype)


def _layout(t, layout):
    """The same values in another memory layout, on the GPU."""
    if layout == "dense":
        return t.cuda()
    if layout == "heads_first":                      # (N, H, L, D) in memory
        return t.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
    if layout == "packed":                           # every third row of a projection
        N, L, H, D = t.shape
        hold = torch.full((N, L, 3, H, D), float("nan"), dtype=t.dtype)
        hold[:, :, 1] = t
        return hold.cuda()[:, :, 1]
    if layout == "shifted":                          # element-aligned base and odd strides
        N, L, H, D = t.shape
        hold = torch.full((N, L, H * D + 1), float("nan"), dtype=t.dtype)
        hold[:, :, 1:] = t.reshape(N, L, H * D)
        return hold.cuda()[:, :, 1:].unflatten(2, (H, D))
    raise ValueError(layout)


class Problem:
    def __init__(self, gs, seed, dtype, N, H, D, q, k, nb=0, causal=False, bias=True,
                 layout="dense", k_len=None, table=None, buckets=None, origin=(0, 0)):
        g = wl.rng(seed)
        self.gs, self.dtype, self.q, self.k = gs, dtype, q, k
        Lq, Lk = q[0] * q[1], k[0] * k[1]
        make = lambda L: _draw(g, (N, L, H, D), dtype)
        self.Q, self.K, self.V = make(Lq), make(Lk), make(Lk)
        self.dO = make(Lq)
        self.scale = 1.0 / math.sqrt(D)
        self.bias = self.which = self.table = self.buckets = None
        if bias:
            m, rows = gs.gs_relative_buckets(q, k, nb, 4 * max(nb, 1), causal, origin, device="cpu")
            self.buckets = m if buckets is None else buckets
            self.table = _draw(g, (rows, H), dtype, 0.7) if table is None else table
            self.bias, self.which = ref.pair_bias(self.table, self.buckets, q, k)
        self.k_len = None if k_len is None else torch.tensor(k_len, dtype=torch.int32)
        self.layout = layout

    def args(self):
        dev = lambda t: None if t is None else t.cuda()
        return dict(table=dev(self.table), buckets=dev(self.buckets), q_extent=self.q,
                    k_extent=self.k, k_len=dev(self.k_len), scale=self.scale)

    def qkv(self):
        return [_layout(t, self.layout) for t in (self.Q, self.K, self.V)]

    def forward(self):
        o, lse, A = ref.attention(self.Q, self.K, self.V, self.scale, self.bias, self.k_len)
        O, LSE = self.gs.gs_attention(*self.qkv(), **self.args())
        ref.check(O, o, A, self.dtype, "O")
        # the maximum and the logarithm: the score's error and fp32 ulps of both
        size = torch.where(torch.isfinite(lse), lse.abs() + 8, torch.zeros_like(lse))
        ref.check(LSE, lse, size, "float32", "LSE")
        return O, LSE

    def backward(self):
        o, lse, _ = ref.attention(self.Q, self.K, self.V, self.scale, self.bias, self.k_len)
        O, LSE = o.to(DT[self.dtype]).contiguous(), lse.float()
        nb = 0 if self.table is None else self.table.shape[0]
        grads, sums = ref.attention_backward(self.dO, self.Q, self.K, self.V, O, LSE, self.scale,
                                             self.bias, self.k_len, self.which, nb)
        call = lambda: self.gs.gs_attention_backward(self.dO.cuda(), *self.qkv(), O.cuda(),
                                                     LSE.cuda(), **self.args())
        got = call()
        assert len(got) == len(grads)
        for name, a, r, A in zip(("dQ", "dK", "dV", "dTable"), got, grads, sums):
            ref.check(a, r, A, self.dtype, name)
        for a, b in zip(got, call()):     # no sum depends on the order of threads
            assert torch.equal(a, b) or torch.isnan(a).any()
        return got

    def both(self):
        self.forward()
        self.backward()
        assert self.gs.gs_device_status() == 0


GRIDS = [  # N, H, D, q_extent, k_extent, buckets per axis (0: one per offset)
    (1, 1, 16, (1, 1), (1, 1), 0),
    (2, 3, 32, (1, 2), (1, 2), 0),
    (1, 2, 64, (1, 127), (1, 127), 32),
    (1, 2, 64, (1, 128), (1, 64), 0),
    (2, 1, 64, (1, 129), (1, 193), 16),
    (1, 1, 128, (1, 300), (1, 257), 8),
    (3, 2, 32, (8, 8), (8, 8), 0),
    (2, 2, 48, (7, 9), (7, 9), 8),
    (1, 2, 64, (12, 20), (12, 20), 16),
    (1, 1, 64, (3, 100), (5, 70), 0),
    (2, 2, 96, (20, 1), (31, 1), 8),
    (1, 3, 24, (2, 65), (2, 65), 0),
    (1, 1, 80, (64, 3), (64, 3), 0),
    (1, 2, 40, (1, 520), (1, 520), 32),
    (2, 4, 64, (1, 1), (1, 700), 32),
    (1, 2, 64, (1, 5), (1, 1500), 32),
    (1, 1, 1, (4, 5), (4, 5), 0),
    (1, 2, 5, (1, 70), (1, 70), 8),
    (2, 1, 20, (1, 33), (3, 33), 0),
    (1, 1, 127, (6, 11), (6, 11), 0),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(GRIDS)))
def test_forward_and_gradient_on_grids(gs_cuda, case, dtype):
    N, H, D, q, k, nb = GRIDS[case]
    Problem(gs_cuda, 100 + case, dtype, N, H, D, q, k, nb).both()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["heads_first", "packed", "shifted"])
@pytest.mark.parametrize("D", [32, 64, 72, 128])
def test_strided_inputs(gs_cuda, layout, D, dtype):
    Problem(gs_cuda, 200 + D, dtype, 2, 3, D, (5, 17), (5, 17), 8, layout=layout).both()


@pytest.mark.parametrize("dtype", DTYPES)
def test_heads_that_share_keys(gs_cuda, dtype):
    p = Problem(gs_cuda, 210, dtype, 2, 4, 64, (1, 90), (1, 150), 16)
    p.K = p.K[:, :, :1].expand(-1, -1, 4, -1)
    p.V = p.V[:, :, :1].expand(-1, -1, 4, -1)
    dense = gs_cuda.gs_attention(*p.qkv(), **p.args())
    shared = gs_cuda.gs_attention(p.Q.cuda(), p.K[:, :, :1].cuda().expand(-1, -1, 4, -1),
                                  p.V[:, :, :1].cuda().expand(-1, -1, 4, -1), **p.args())
    o, lse, A = ref.attention(p.Q, p.K, p.V, p.scale, p.bias)
    for O, _ in (dense, shared):
        ref.check(O, o, A, dtype, "O")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("q,k", [((1, 70), (1, 70)), ((9, 13), (9, 13)), ((1, 200), (1, 330))])
def test_without_bias(gs_cuda, q, k, dtype):
    Problem(gs_cuda, 220, dtype, 2, 2, 64, q, k, bias=False).both()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[0, 1, 200], [64, 63, 65], [128, 199, 129], [-5, 1000, 7]])
@pytest.mark.parametrize("D", [64, 20])
def test_ragged_lengths(gs_cuda, lens, D, dtype):
    Problem(gs_cuda, 230, dtype, 3, 2, D, (10, 20), (10, 20), 8, k_len=lens).both()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Lq", [1, 3])
def test_single_tokens_over_ragged_memory(gs_cuda, Lq, dtype):
    Problem(gs_cuda, 240, dtype, 4, 2, 64, (1, Lq), (1, 3001), 32, k_len=[0, 1, 1500, 3001],
            origin=(0, 3001 - Lq)).both()


@pytest.mark.parametrize("dtype", DTYPES)
def test_what_masked_keys_hold_is_never_used(gs_cuda, dtype):
    lens = [37, 0, 150]
    p = Problem(gs_cuda, 250, dtype, 3, 2, 64, (1, 150), (1, 150), 16, k_len=lens)
    O, LSE = p.forward()
    G = p.backward()
    for n, m in enumerate(lens):
        p.K[n, m:] = float("nan")
        p.V[n, m:] = float("inf")
    O2, LSE2 = gs_cuda.gs_attention(*p.qkv(), **p.args())
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    for a, b in zip(G, p.backward()):
        assert torch.equal(a, b)
    one = Problem(gs_cuda, 251, dtype, 2, 2, 64, (1, 1), (1, 900), 16, k_len=[100, 333])
    O, LSE = one.forward()
    one.K[0, 100:], one.V[0, 100:], one.V[1, 333:] = float("inf"), float("nan"), float("nan")
    O2, LSE2 = gs_cuda.gs_attention(*one.qkv(), **one.args())
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 36])
@pytest.mark.parametrize("Lq,Lk", [(1, 1), (140, 140), (300, 300), (130, 260)])
def test_causal_bucket_map(gs_cuda, Lq, Lk, D, dtype):
    p = Problem(gs_cuda, 260, dtype, 2, 2, D, (1, Lq), (1, Lk), 16, causal=True)
    p.both()


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_without_any_key(gs_cuda, dtype):
    # offsets in a window only, and a table row of -inf: many queries keep no key
    q, k = (1, 150), (1, 150)
    off = torch.arange(299) - 149
    buckets = torch.where((off >= 100) & (off < 120), off - 100, -7).to(torch.int32)
    buckets[149 + 110] = 99                                # beyond the table
    g = wl.rng(270)
    table = _draw(g, (20, 2), dtype, 0.7)
    table[3] = float("-inf")
    p = Problem(gs_cuda, 271, dtype, 2, 2, 64, q, k, table=table, buckets=buckets)
    O, LSE = p.forward()
    assert not O[:, :100].any() and torch.isinf(LSE[:, :, :100]).all()
    dQ, dK, dV, dT = p.backward()
    assert not dQ[:, :100].any() and not dK[:, 50:].any() and not dT[3].any()
    assert gs_cuda.gs_device_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_lowest_finite_entries_are_an_ordinary_softmax(gs_cuda, dtype):
    # every pair of some offsets at the type's lowest value: alone in a row they share it evenly
    low = torch.finfo(DT[dtype]).min
    q, k = (1, 80), (1, 80)
    off = torch.arange(159) - 79
    buckets = torch.where(off < 0, 0, 1).to(torch.int32)   # keys after the query: entry 0
    table = torch.tensor([[low], [0.25]], dtype=DT[dtype])
    p = Problem(gs_cuda, 280, dtype, 1, 1, 64, q, k, table=table, buckets=buckets)
    O, _ = gs_cuda.gs_attention(*p.qkv(), **p.args())
    o, _, A = ref.attention(p.Q, p.K, p.V, p.scale, p.bias)
    ref.check(O, o, A, dtype, "O")
    p.table[1] = low
    # with one common entry the scores survive only as far as the type's lowest value keeps them
    # in fp32 (fp16's does, by 2^-8 a step), so the row is a softmax of nearly equal scores
    O, LSE = gs_cuda.gs_attention(*p.qkv(), **p.args())
    assert torch.isfinite(O).all() and torch.isfinite(LSE).all()
    if dtype != "float16":
        mean = p.V.double().mean(1, keepdim=True).expand(-1, 80, -1, -1)
        ref.check(O, mean, p.V.double().abs().mean(1, keepdim=True).expand(-1, 80, -1, -1), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_far_apart_and_growing(gs_cuda, dtype):
    # scores that rise along the keys make the running maximum move at every tile
    p = Problem(gs_cuda, 290, dtype, 1, 2, 64, (1, 140), (1, 400), bias=False)
    ramp = torch.linspace(-6, 6, 400).view(1, 400, 1, 1)
    p.Q = torch.ones_like(p.Q)
    p.K = (p.K.float() * 0.1 + ramp).to(p.K.dtype)
    O, _ = p.gs.gs_attention(*p.qkv(), **p.args())
    o, _, A = ref.attention(p.Q, p.K, p.V, p.scale)
    # scores reach 48: their fp32 error, and the weight's, doubles against the derivation
    ref.check(O, o, A, dtype, "O", C=512.0)


def test_non_finite_values_stay_in_their_rows(gs_cuda):
    for dtype in DTYPES:
        p = Problem(gs_cuda, 300, dtype, 1, 1, 64, (1, 200), (1, 200), 16)
        O, LSE = gs_cuda.gs_attention(*p.qkv(), **p.args())
        p.Q[0, 5, 0, 3] = float("nan")
        O2, LSE2 = gs_cuda.gs_attention(*p.qkv(), **p.args())
        assert torch.isnan(O2[0, 5]).all() and torch.isnan(LSE2[0, 0, 5])
        keep = torch.arange(200, device="cuda") != 5
        assert torch.equal(O2[:, keep], O[:, keep])


def test_gradient_against_differences(gs_cuda):
    p = Problem(gs_cuda, 310, "float32", 2, 2, 24, (5, 7), (5, 7), 8, k_len=[35, 20])
    dQ, dK, dV, dT = (t.double().cpu() for t in p.backward())
    q, k, v, t = p.Q.double(), p.K.double(), p.V.double(), p.table.double()
    w = p.dO.double()

    def f(q_, k_, v_, t_):
        bias, _ = ref.pair_bias(t_, p.buckets, p.q, p.k)
        return (ref.attention(q_, k_, v_, p.scale, bias, p.k_len)[0] * w).sum()

    g, h = wl.rng(311), 1e-5
    for _ in range(4):
        d = [torch.from_numpy(g.normal(size=x.shape)) for x in (q, k, v, t)]
        up = f(*(x + h * y for x, y in zip((q, k, v, t), d)))
        down = f(*(x - h * y for x, y in zip((q, k, v, t), d)))
        parts = [(a * y) for a, y in zip((dQ, dK, dV, dT), d)]
        size = sum(x.abs().sum() for x in parts)
        # central differences: h^2 f'''/6 + 1e-16 f / h ~ 1e-9; fp32 O and LSE: 1e-6
        assert abs((up - down) / (2 * h) - sum(x.sum() for x in parts)) <= 1e-5 * size


def test_empty_extents(gs_cuda):
    Q = torch.empty((2, 0, 2, 64), device="cuda")
    K = torch.randn((2, 5, 2, 64), device="cuda")
    O, LSE = gs_cuda.gs_attention(Q, K, K)
    assert O.numel() == 0 and LSE.shape == (2, 2, 0)
    dQ, dK, dV = gs_cuda.gs_attention_backward(Q, Q, K, K, O, LSE)
    assert dQ.shape == Q.shape and not dK.any() and not dV.any()
    Q = torch.randn((2, 5, 2, 64), device="cuda")
    K = torch.empty((2, 0, 2, 64), device="cuda")
    O, LSE = gs_cuda.gs_attention(Q, K, K)
    assert not O.any() and (LSE == float("-inf")).all()
    dQ, dK, dV = gs_cuda.gs_attention_backward(Q, Q, K, K, O, LSE)
    assert not dQ.any() and dK.numel() == 0


def test_runs_on_the_current_stream_and_in_a_graph(gs_cuda):
    p = Problem(gs_cuda, 320, "bfloat16", 2, 2, 64, (6, 30), (6, 30), 8)
    args, (Q, K, V) = p.args(), p.qkv()
    dO = p.dO.cuda()
    want = gs_cuda.gs_attention(Q, K, V, **args)
    grads = gs_cuda.gs_attention_backward(dO, Q, K, V, *want, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O, LSE = gs_cuda.gs_attention(Q, K, V, **args)
        again = gs_cuda.gs_attention_backward(dO, Q, K, V, O, LSE, **args)
    O.zero_()
    for t in again:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, want[0]) and torch.equal(LSE, want[1])
    for a, b in zip(again, grads):
        assert torch.equal(a, b)


def test_offsets_beyond_32_bits(gs_cuda):
    # a memory whose last head rows lie more than 2^32 bytes and 2^31 elements from its start
    N, L, H, D = 1, 70000, 512, 64
    kv = torch.zeros((N, L, H, D), dtype=torch.bfloat16, device="cuda")
    assert kv.numel() > 1 << 31
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    tail = torch.randn((N, 300, 2, D), generator=g, device="cuda").to(torch.bfloat16)
    kv[:, L - 300:, H - 2:] = tail
    for Lq in (1, 130):
        Q = torch.randn((N, Lq, 2, D), generator=g, device="cuda").to(torch.bfloat16)
        far = kv[:, L - 300:, H - 2:]
        O, LSE = gs_cuda.gs_attention(Q, far, far)
        whole, _ = gs_cuda.gs_attention(Q, kv[:, :, H - 2:], kv[:, :, H - 2:])
        o, lse, A = ref.attention(Q, tail, tail, D ** -0.5)
        ref.check(O, o, A, "bfloat16", "O")
        keys = torch.cat([torch.zeros((N, L - 300, 2, D), dtype=torch.bfloat16, device="cuda"),
                          tail], 1)
        o, lse, A = ref.attention(Q, keys, keys, D ** -0.5)
        ref.check(whole, o, A, "bfloat16", "whole")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_many_tiles_give_the_same_bits_every_time(gs_cuda, dtype):
    # thousands of blocks whose warps drift apart over 64 key tiles: a wait that lets one warp
    # read a sum too early shows as a run that differs
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    q, k = (16, 64), (64, 64)
    m, rows = gs_cuda.gs_relative_buckets(q, k, 16, 64)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])
    Q, K, V, table = mk(16, 1024, 8, 64), mk(16, 4096, 8, 64), mk(16, 4096, 8, 64), mk(rows, 8)
    call = lambda: gs_cuda.gs_attention(Q, K, V, table, m, q, k)
    O, LSE = call()
    for _ in range(12):
        O2, LSE2 = call()
        assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    for n, h in ((0, 0), (15, 7)):   # two heads in full
        bias, _ = ref.pair_bias(table[:, h:h + 1], m, q, k)
        o, lse, A = ref.attention(Q[n:n + 1, :, h:h + 1], K[n:n + 1, :, h:h + 1],
                                  V[n:n + 1, :, h:h + 1], 0.125, bias)
        ref.check(O[n:n + 1, :, h:h + 1], o, A, dtype, "O")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("q,k", [((3, 400), (3, 400)), ((2, 700), (3, 700)), ((300, 2), (150, 4))])
def test_grids_whose_rows_end_inside_tiles(gs_cuda, q, k, dtype):
    # the relative indices of one tile then lie far apart
    Problem(gs_cuda, 330, dtype, 1, 1, 32, q, k, 16).both()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gradient_of_many_tiles_gives_the_same_bits_every_time(gs_cuda, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(10)
    q = k = (32, 64)
    m, rows = gs_cuda.gs_relative_buckets(q, k, 16, 64)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dtype])
    Q, K, V, dO = (mk(8, 2048, 8, 64) for _ in range(4))
    table = mk(rows, 8)
    k_len = torch.tensor([2048, 2000, 1, 64, 1024, 2047, 700, 65], dtype=torch.int32, device="cuda")
    args = (table, m, q, k, k_len)
    O, LSE = gs_cuda.gs_attention(Q, K, V, *args)
    call = lambda: gs_cuda.gs_attention_backward(dO, Q, K, V, O, LSE, *args)
    first = call()
    for _ in range(8):
        for a, b in zip(first, call()):
            assert torch.equal(a, b)
    for n, h in ((1, 0), (7, 5)):    # two heads in full; the table's gradient takes all of them
        one = lambda t: t[n:n + 1, :, h:h + 1]
        bias, which = ref.pair_bias(table[:, h:h + 1], m, q, k)
        grads, sums = ref.attention_backward(one(dO), one(Q), one(K), one(V), one(O),
                                             LSE[n:n + 1, h:h + 1], 0.125, bias, k_len[n:n + 1])
        for name, a, r, A in zip(("dQ", "dK", "dV"), first, grads, sums):
            ref.check(one(a), r, A, dtype, name)


def test_bias_gradient_summed_over_several_launches(gs_cuda):
    # 68 heads of 64 x 64 tokens: more partial sums than one launch keeps
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    N, H, q = 4, 17, (64, 64)
    m, rows = gs_cuda.gs_relative_buckets(q, q, 16, 64)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").half()
    Q, K, V, dO = (mk(N, 4096, H, 16) for _ in range(4))
    table = mk(rows, H)
    O, LSE = gs_cuda.gs_attention(Q, K, V, table, m, q, q)
    dT = gs_cuda.gs_attention_backward(dO, Q, K, V, O, LSE, table, m, q, q)[3].double()
    parts = [gs_cuda.gs_attention_backward(dO[n:n + 1], Q[n:n + 1], K[n:n + 1], V[n:n + 1],
                                           O[n:n + 1], LSE[n:n + 1], table, m, q, q)[3].double()
             for n in range(N)]
    # each side rounds to fp16: half an ulp of every part and of the whole; fp32 sums of 2^24
    # pairs beside it, far below the smallest of those
    lim = ref.U["float16"] / 2 * (dT.abs() + sum(p.abs() for p in parts)) * 1.1 + 1e-2
    assert ((dT - sum(parts)).abs() <= lim).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [32, 96])
@pytest.mark.parametrize("q", [(6, 11), (8, 8), (1, 150)])
def test_many_small_heads_of_ragged_length(gs_cuda, q, D, dtype):
    # several items of work per block, of one to three key tiles, some with no key at all
    L, N = q[0] * q[1], 260
    g = wl.rng(340)
    lens = g.integers(0, L + 1, size=N)
    lens[:4] = [0, L, 1, 0]
    lens[-1] = 0
    Problem(gs_cuda, 341, dtype, N, 3, D, q, q, 8, k_len=[int(x) for x in lens]).both()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Lq", [1, 5, 8])
@pytest.mark.parametrize("D", [4, 8, 16, 128])
def test_few_queries_at_every_width_of_a_key(gs_cuda, D, Lq, dtype):
    # from one lane per key to a whole warp, keys shared by up to sixteen blocks
    Problem(gs_cuda, 440, dtype, 1, 3, D, (1, Lq), (3, 811), 16, k_len=[2200]).forward()
    Problem(gs_cuda, 441, dtype, 2, 2, D, (1, Lq), (1, 131)).forward()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [40, 64, 77, 128])
@pytest.mark.parametrize("q,k", [((1, 9), (1, 2050)), ((1, 130), (1, 1023)), ((3, 20), (4, 211))])
def test_long_keys_shared_by_the_blocks_of_a_cluster(gs_cuda, q, k, D, dtype):
    # lengths that leave some blocks a part of a tile, one key or nothing
    Lk = k[0] * k[1]
    p = Problem(gs_cuda, 450, dtype, 6, 2, D, q, k, 16, k_len=[Lk, 0, 1, 65, 513, Lk - 63])
    O, LSE = p.forward()
    O2, LSE2 = gs_cuda.gs_attention(*p.qkv(), **p.args())
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    Problem(gs_cuda, 451, dtype, 1, 1, D, q, k, bias=False, layout="packed").forward()
    # masked by the map: whole tiles, and with them whole blocks, that hold no key
    Problem(gs_cuda, 452, dtype, 1, 2, D, (1, 140), (1, Lk), 16, causal=True).forward()
    assert gs_cuda.gs_device_status() == 0
