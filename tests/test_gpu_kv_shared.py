"""Attention of requests that share prefixes, against the definition in 64 bits
(error bounds: kv_common.bounds and round_common.small_weights)."""
import numpy as np
import pytest
import torch

import gpu_common as gc
import kv_common as kc
import round_common as rc

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
PAGE, LENGTH = 12, 13


@pytest.fixture(scope="module")
def ssdv():
    return gc.cuda_lib()


class Groups:
    """Requests in groups: a prefix each, in shared pages as far as it fills them, then the requests' own tokens."""

    def __init__(self, ssdv, sizes, pre, own, n, Hkv, G, D, page, dtype, n_q=None, past_only=False, seed=1, edit=None,
                 q_size=1.0):
        self.ssdv, self.n, self.G, self.D, self.page, self.dtype, self.past_only = ssdv, n, G, D, page, dtype, past_only
        self.start = np.concatenate([[0], np.cumsum(sizes)])
        self.pre, self.B = np.asarray(pre), int(self.start[-1])
        group = np.repeat(np.arange(len(sizes)), sizes)
        self.group = group
        own = np.asarray(own)
        self.lens = self.pre[group] + own
        self.nq = np.full(self.B, n) if n_q is None else np.asarray(n_q)
        self.n_q = n_q
        count = self.lens if past_only else self.lens + self.nq
        T = int(max(1, count.max()))
        k, k64 = kc.rows((self.B, T, Hkv, D), dtype, seed)
        v, v64 = kc.rows((self.B, T, Hkv, D), dtype, seed + 1)
        first = self.start[:-1][group]
        for b in range(self.B):  # every request holds its group's prefix
            m = int(self.pre[group[b]])
            for x, y in ((k, k), (v, v), (k64, k64), (v64, v64)):
                x[b, :m] = y[int(first[b]), :m]
        self.q, self.q64 = kc.rows((self.B, n, Hkv * G, D), dtype, seed + 2, q_size)
        if edit is not None:
            edit(self, k, v)
            k64, v64 = k.double().cpu().numpy(), v.double().cpu().numpy()
        self.width = max(1, -(-(int(self.lens.max()) + n) // page))
        g = np.random.default_rng(seed)
        self.cache = ssdv.make_kv_cache(self.B * self.width + 3, Hkv, D, page, device="cuda")
        self.cache.fill_(0xFF)
        table = g.permutation(self.B * self.width + 3)[:self.B * self.width].reshape(self.B, self.width)
        self.full = self.pre[group] // page
        for b in range(self.B):
            table[b, :self.full[b]] = table[int(first[b]), :self.full[b]]
        self.table = kc.ints(table)
        begin = np.where(np.arange(self.B) == first, 0, self.full * page)
        longest = max(1, int((count - begin).max()))
        mine_k, mine_v = k.new_zeros((self.B, longest) + k.shape[2:]), v.new_zeros((self.B, longest) + v.shape[2:])
        for b in range(self.B):
            m = int(count[b] - begin[b])
            mine_k[b, :m], mine_v[b, :m] = k[b, begin[b]:count[b]], v[b, begin[b]:count[b]]
        ssdv.kv_append(self.cache, self.table, kc.ints(begin), mine_k, mine_v, n_new=kc.ints(count - begin))
        self.kh, self.vh = kc.held(k64), kc.held(v64)

    def run(self, status=0, **kw):
        H = self.q.shape[2]
        args = dict(start=kc.ints(self.start), shared=kc.ints(self.pre), q=self.q, scale=None)
        args.update(kw)
        ws = torch.zeros(self.ssdv.kv_shared_workspace_bytes(self.B, self.n, H, H // self.G, self.D, args["shared"].numel()),
                         dtype=torch.uint8, device="cuda")
        ws[16:].fill_(0xFF)
        out, lse = self.ssdv.kv_attention_shared(
            self.cache, self.table, kc.ints(self.lens), args["q"], args["start"], args["shared"],
            n_q=None if self.n_q is None else kc.ints(self.nq), scale=args["scale"], past_only=self.past_only,
            return_lse=True, workspace=ws)
        assert self.ssdv.read_status(ws) == status
        return out, lse

    def compare(self, out, lse, scale=None, only=None):
        scale = self.D ** -0.5 if scale is None else scale
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(self.B) if only is None else only:
            def seen(i):
                return np.arange(0 if i >= self.nq[b] else self.lens[b] if self.past_only else self.lens[b] + i + 1)
            ref, every = rc.attend(self.q64[b], self.kh[b], self.vh[b], seen, scale)
            tol, ltol = kc.bounds(*ref, self.D, self.dtype)
            tol = tol + rc.small_weights(every, self.dtype)
            gone = ref[4] == 0
            assert (out[b][gone] == 0).all() and (lse[b][gone] == -np.inf).all(), b
            err = np.abs(out[b] - ref[0])
            assert (err <= tol)[~gone].all(), (b, float(np.nanmax(err / tol)), int(np.isnan(err).sum()))
            lerr = np.abs(lse[b][~gone] - ref[1][~gone])
            assert (lerr <= ltol[~gone]).all(), (b, float((lerr / ltol[~gone]).max()))


def check(ssdv, *args, **kw):
    g = Groups(ssdv, *args, **kw)
    g.compare(*g.run())
    return g


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hkv,G,n", [(1, 1, 1), (2, 4, 5), (3, 3, 2), (1, 16, 9), (2, 8, 1)])
def test_shapes(ssdv, Hkv, G, n, D, dtype):
    check(ssdv, [3, 1, 2], [70, 0, 129], [5, 40, 0, 17, 1, 64], n, Hkv, G, D, 16, dtype)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_prefix_lengths(ssdv, dtype, D):
    """Prefixes that end around a block, a page and a tile's end, none and one token among them."""
    pre = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400]
    own = [(7 * b) % 23 for b in range(2 * len(pre))]
    for page, past_only in ((16, False), (48, True), (128, False)):
        check(ssdv, [2] * len(pre), pre, own, 3, 1, 4, D, page, dtype, past_only=past_only)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 128)])
@pytest.mark.parametrize("size", [1, 7, 8, 9, 31, 32, 33, 64, 65, 100])
def test_group_sizes(ssdv, size, dtype, D):
    """Row blocks that are empty, partly filled and full: 1 to 600 rows a kv head."""
    g = np.random.default_rng(size)
    check(ssdv, [size, 2], [200, 30], g.integers(0, 40, size + 2), 2, 1, 3, D, 16, dtype)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ragged_queries(ssdv, D, dtype):
    n_q = [9, 0, 4, 1, 0, 0, 7]
    for past_only in (False, True):
        check(ssdv, [4, 2, 1], [140, 33, 0], [0, 3, 50, 7, 9, 0, 0], 9, 2, 4, D, 32, dtype, n_q=n_q, past_only=past_only)


@pytest.mark.parametrize("dtype,D,G", [(BF16, 128, 4), (BF16, 64, 2), (BF16, 256, 2), (F32, 64, 2)])
def test_long_prefix(ssdv, dtype, D, G):
    """A prefix that many teams share, of one group and of two."""
    check(ssdv, [9], [6001], np.arange(9) * 11, 3, 1, G, D, 64, dtype)
    check(ssdv, [3, 2], [3000, 2049], np.arange(5), 2, 2, G, D, 64, dtype)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_many_groups(ssdv, dtype, D):
    """More groups than a CTA has threads, empty ones among them, each of few requests."""
    g = np.random.default_rng(3)
    sizes = g.integers(0, 2, 900)
    sizes[0], sizes[-1] = 0, 0
    B = int(sizes.sum())
    check(ssdv, sizes, g.integers(0, 70, 900), g.integers(0, 30, B), 1, 1, 2, D, 16, dtype)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 128)])
@pytest.mark.parametrize("scale,q_size", [(0.0, 1.0), (-0.3, 1.0), (3.0, 4.0), (1e-3, 1e3), (1.0, 1e-30)])
def test_scales(ssdv, scale, q_size, dtype, D):
    """Uniform weights, negative scale, scores in the thousands (one token decides), queries far from one."""
    g = Groups(ssdv, [5, 2], [300, 40], [3, 0, 50, 20, 9, 8, 1], 3, 1, 4, D, 16, dtype, q_size=q_size)
    g.compare(*g.run(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_first_tokens_draw_the_weight(ssdv, dtype, D):
    """Large scores and values of zero at the first tokens: what remains are small weights."""
    def edit(g, k, v):
        for b in range(g.B):
            k[b, :2], v[b, :2] = g.q[int(g.start[g.group[b]]), 0, :2] * 2, 0
    check(ssdv, [4, 3], [700, 333], np.arange(7) * 9, 2, 2, 4, D, 16, dtype, edit=edit)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (BF16, 256), (F32, 64)])
def test_rising_scores(ssdv, dtype, D):
    """Scores that rise along the prefix, a little and a lot: the reference moves with them."""
    for step in (0.002, 0.05):
        def edit(g, k, v):
            at = torch.arange(k.shape[1], device="cuda").float()[None, :, None, None] * step
            k[:] = (k.float() * 0.1 + at * g.q[:1, :1, :1].float() / g.q[0, 0, 0].float().square().sum().sqrt()).to(k.dtype)
        check(ssdv, [4, 3], [900, 333], np.arange(7) * 9, 2, 1, 4, D, 16, dtype, edit=edit)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_query_strides(ssdv, dtype):
    g = Groups(ssdv, [3, 1], [150, 20], [4, 60, 0, 9], 5, 2, 4, 128, 16, dtype)
    flat = torch.zeros(g.q.numel() + 1, dtype=dtype, device="cuda")
    odd = flat[1:].view(g.q.shape).copy_(g.q)
    wide = flat.new_zeros(4, 5, 3, 8, 128)
    wide[:, :, 1] = g.q
    for form in (odd, wide[:, :, 1], g.q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)):
        g.compare(*g.run(q=form))


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (BF16, 256), (F32, 64)])
def test_nan(ssdv, dtype, D):
    """A NaN in the prefix is its whole group's; behind a request's last query it is nobody's, and neither are the bytes
    behind the prefix in its last block (which hold NaN here)."""
    def edit(g, k, v):
        v[:2, 77] = float("nan")
        k[2:4, 3] = float("nan")
    g = Groups(ssdv, [2, 2, 2], [150, 30, 100], [4, 60, 0, 9, 20, 0], 3, 1, 4, D, 16, dtype, edit=edit)
    out, lse = g.run()
    assert torch.isnan(out[:2, ..., 16 * 0:16]).any() and torch.isnan(out[2:4]).all() and torch.isnan(lse[2:4]).all()
    g.compare(out, lse, only=[4, 5])


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_bad_pages(ssdv, dtype, D):
    g = Groups(ssdv, [2, 2], [150, 64], [40, 60, 5, 9], 3, 1, 4, D, 16, dtype, n_q=[3, 2, 3, 3])
    table = g.table.clone()
    for bad in (-1, 1 << 30):
        g.table[0, 4] = bad  # of the prefix, in the first request's row
        out, lse = g.run(status=PAGE)
        assert torch.isnan(out[0]).all() and torch.isnan(out[1, :2]).all() and (out[1, 2] == 0).all()
        g.compare(out, lse, only=[2, 3])
        g.table.copy_(table)
        g.table[1, 4] = bad  # nobody looks there
        g.compare(*g.run())
        g.table.copy_(table)
        g.table[1, 12] = bad  # request 1's own
        out, lse = g.run(status=PAGE)
        assert torch.isnan(out[1, :2]).all()
        g.compare(out, lse, only=[0, 2, 3])
        g.table.copy_(table)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_bad_lengths(ssdv, dtype, D):
    def fresh():
        return Groups(ssdv, [2, 2], [150, 64], [40, 60, 5, 9], 3, 1, 4, D, 16, dtype)
    g = fresh()
    for bad in (-1, 1 << 30, 191):  # 191: longer than request 0, not than request 1
        out, lse = g.run(status=LENGTH, shared=kc.ints([bad, 64]))
        assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all() and (bad == 191 or torch.isnan(out[1]).all())
        g.compare(out, lse, only=[2, 3])
    for start in ([1, 2, 4], [0, 2, 3], [0, 2, 5], [0, 5, 4], [0, -1, 4], [0, 3, 2]):
        out, lse = g.run(status=LENGTH, start=kc.ints(start))
        assert torch.isnan(out).all() and torch.isnan(lse).all(), start
    g.lens[1] = -5
    out, lse = g.run(status=LENGTH)
    assert torch.isnan(out[1]).all()
    g.compare(out, lse, only=[0, 2, 3])


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_the_same_as_one_by_one(ssdv, dtype, D):
    """Groups of one request, and prefixes of nothing, are plain attention; repeats give the same bits."""
    g = Groups(ssdv, [5], [200], [1, 30, 0, 77, 150], 4, 2, 4, D, 16, dtype)
    a = g.run()
    b = g.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    g.compare(*a)
    g.compare(*g.run(start=kc.ints(np.arange(6)), shared=kc.ints(g.lens)))
    g.compare(*g.run(start=kc.ints(np.arange(6)), shared=kc.ints([0] * 5)))
    g.compare(*g.run(shared=kc.ints([0])))
    g.compare(*g.run(start=kc.ints([0, 2, 2, 5]), shared=kc.ints([200, 9, 16])))


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_capture_streams_and_growth(ssdv, dtype, D):
    """Two captured graphs keep workspaces of their own; lengths and groups are read at each replay."""
    g = Groups(ssdv, [3, 2], [300, 40], [9, 9, 20, 5, 0], 3, 1, 4, D, 16, dtype)
    start, shared, lens = kc.ints(g.start), kc.ints(g.pre), kc.ints(g.lens)
    call = lambda: ssdv.kv_attention_shared(g.cache, g.table, lens, g.q, start, shared, return_lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call()
    torch.cuda.current_stream().wait_stream(side)
    g.compare(*other)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call())
        graphs.append(graph)
    for _ in range(3):
        for s, graph in zip((side, torch.cuda.current_stream()), graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            g.compare(*out)
    shared.copy_(kc.ints([100, 0]))
    start.copy_(kc.ints([0, 3, 5]))
    graphs[0].replay()
    g.compare(*outs[0])


@pytest.mark.parametrize("dtype,D,G,n", [(BF16, 64, 128, 32), (BF16, 128, 60, 5), (F32, 64, 128, 32)])
def test_requests_of_more_rows_than_a_block(ssdv, dtype, D, G, n):
    """A request's rows, 300 to 4096 a kv head, lie in several row blocks, some of which other requests share."""
    check(ssdv, [2, 1], [50, 20], [0, 3, 1], n, 1, G, D, 16, dtype)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_pages_far_into_a_large_pool(ssdv, dtype, D):
    """Blocks beyond 4 GiB, some of the pool's last pages."""
    g = Groups(ssdv, [3, 2], [200, 90], [9, 0, 40, 5, 30], 2, 1, 4, D, 64, dtype)
    far = (5 << 30) // g.cache[0].numel()
    pool = torch.empty((far + g.cache.shape[0],) + tuple(g.cache.shape[1:]), dtype=torch.uint8, device="cuda")
    pool[far:] = g.cache
    g.cache = pool
    g.table += far
    g.compare(*g.run())


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_two_streams_at_once(ssdv, dtype, D):
    """Calls on two streams, each with the workspace of its stream, many times over."""
    a = Groups(ssdv, [6], [900], np.arange(6) * 20, 3, 2, 4, D, 16, dtype, seed=1)
    b = Groups(ssdv, [2, 4], [300, 700], np.arange(6) * 11, 3, 2, 4, D, 32, dtype, seed=5)
    args = [(kc.ints(g.lens), kc.ints(g.start), kc.ints(g.pre)) for g in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for g, (lens, start, shared), s in zip((a, b), args, streams):
            with torch.cuda.stream(s):
                outs.append(ssdv.kv_attention_shared(g.cache, g.table, lens, g.q, start, shared, return_lse=True))
    torch.cuda.synchronize()
    a.compare(*outs[0])
    b.compare(*outs[1])
    for x, y in zip(outs, outs[2:]):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("D", [64, 128])
def test_a_bad_query_is_its_own_rows_loss(ssdv, D):
    """NaN and infinite queries beside others of the same row block."""
    g = Groups(ssdv, [4], [300], [3, 9, 0, 20], 2, 1, 4, D, 16, BF16)
    q = g.q.clone()
    q[1, 0, 2, 5], q[2, 1, 0, 7] = float("nan"), float("inf")
    out, lse = g.run(q=q)
    assert torch.isnan(out[1, 0, 2]).all() and torch.isnan(out[2, 1, 0]).all()
    out[1, 0, 2], lse[1, 0, 2], out[2, 1, 0], lse[2, 1, 0] = g.run()[0][1, 0, 2], g.run()[1][1, 0, 2], g.run()[0][2, 1, 0], \
        g.run()[1][2, 1, 0]
    g.compare(out, lse)
