"""A layer's step as it is used: the cache append, the block scores, the
selection and the attention over the selected blocks, one after the other on
one stream, against the oracles; the new entry points captured into a graph
and replayed, called from several threads at once, on another stream, and with
keys past 4 GiB."""
import sys
import threading

import pytest
import torch

import layer_cases as lc
import oracle
from oracle import layer
from test_append_gpu import angles
from test_attention_gpu import call, check, to

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_max_qk_amd
    block_max_qk_amd.load_library()
    return torch.device("cuda:0")


class Layer:
    """Caches of one layer and its step; the index branch in `kind`."""

    def __init__(self, kind, layout, B, MB, dev, dtype=FP):
        self.kind, self.layout, self.dev, self.dtype = kind, layout, dev, dtype
        gen = torch.Generator().manual_seed(5)
        pages = B * MB + 1
        self.table = torch.randperm(pages, generator=gen)[:B * MB].view(B, MB).int().to(dev)
        zeros = lambda H, last, dt: torch.zeros(lc.cache_shape(layout, pages, H, last), dtype=dt,  # noqa: E731
                                                device=dev)
        self.k, self.v = zeros(2, 128, dtype), zeros(2, 128, dtype)
        self.scale = None
        if kind == "mxfp4":
            self.ik, self.scale = zeros(1, 64, torch.uint8), zeros(1, 4, torch.uint8)
        elif kind == "i8":
            self.ik, self.scale = zeros(1, 128, torch.int8), torch.zeros(pages, 1, 128, device=dev)
        else:
            self.ik = zeros(1, 128, torch.float8_e4m3fn if kind == "e4m3" else dtype)
        cos, sin = angles(MB * 128, 64)
        self.cos, self.sin = cos.to(dev), sin.to(dev)

    def step(self, x, cu, kv, k=3):
        """x [T, 8 + 2 + 2 + 2 + 1, 128]: queries, keys, values, index queries
        (one per KV head) and the index key."""
        import block_max_qk_amd as m
        T, MB = x.shape[0], self.table.shape[1]
        q = torch.empty(T, 8, 128, dtype=self.dtype, device=self.dev)
        iq_scale = None
        if self.kind == "mxfp4":
            iq = torch.empty(T, 2, 64, dtype=torch.uint8, device=self.dev)
            iq_scale = torch.empty(T, 2, 4, dtype=torch.uint8, device=self.dev)
        else:
            it = torch.float8_e4m3fn if self.kind == "e4m3" else self.dtype
            iq = torch.empty(T, 2, 128, dtype=it, device=self.dev)
        m.msa_cache_append([m.CacheItem(x[:, :8], q, "ROWS", rotate=True),
                            m.CacheItem(x[:, 8:10], self.k, self.layout, rotate=True),
                            m.CacheItem(x[:, 10:12], self.v, self.layout),
                            m.CacheItem(x[:, 12:14], iq, "ROWS", iq_scale, True),
                            m.CacheItem(x[:, 14:], self.ik, self.layout, self.scale, True)],
                           self.cos, self.sin, self.table, cu, kv)
        W = m.msa_index_score_out_width(MB)
        scores = torch.empty(2, T, W, device=self.dev)
        if self.kind == "mxfp4":
            m.msa_index_score_mxfp4(iq, iq_scale, self.ik, self.scale, None, self.table, cu, kv,
                                    self.layout, 3, 1, 1, scores, MB, local_mode="query")
        else:
            m.msa_index_score(iq, self.ik, None, self.table, self.scale, cu, kv, self.layout, 3, 1,
                              1, scores, MB, local_mode="query")
        blocks = m.block_topk(scores, MB, k)
        out, lse = m.block_attention(q, self.k, self.v, blocks, self.table, cu, kv, self.layout,
                                     return_lse=True)
        return q, scores, blocks, out, lse


@pytest.mark.parametrize("kind,layout,dtype", [("same", "BBND", BF), ("e4m3", "BBND", FP),
                                               ("i8", "BNBD", FP), ("mxfp4", "BNBD", BF)])
def test_steps_of_a_layer(kind, layout, dtype, dev):
    """A prompt chunk, then two decode steps, each checked: the caches by the
    append's tests, here the scores' selection and the attention on the caches
    as they are."""
    log("layer", kind, layout)
    L = Layer(kind, layout, 3, 8, dev, dtype)
    gen = torch.Generator().manual_seed(6)
    kv = torch.zeros(3, dtype=torch.int32)
    for q_lens in ([300, 1, 700], [1, 1, 1], [1, 3, 2]):
        cu, T = lc.lengths(q_lens)
        kv = kv + torch.tensor(q_lens, dtype=torch.int32)
        x = torch.randn(T, 15, 128, generator=gen).to(dtype)
        q, scores, blocks, out, lse = L.step(x.to(dev), cu.to(dev), kv.to(dev))
        torch.cuda.synchronize()
        assert torch.equal(blocks.cpu(), oracle.block_topk(scores.cpu(), 8, 3))
        c = {"q": q.cpu(), "k": L.k.cpu(), "v": L.v.cpu(), "table": L.table.cpu(), "cu": cu,
             "kv": kv, "layout": layout, "mode": 3, "blocks": blocks.cpu()}
        check(c, out, lse)
        # every token sees its own key among the selected ones
        own = torch.tensor([p // 128 for _, _, p in layer.positions(cu, kv, T)])
        assert (blocks.cpu() == own[:, None, None]).any(-1).all()


def _entries(dev):
    import block_max_qk_amd as m
    work = []
    for name, c in (("rows split", lc.attention_case([1, 1], [3000, 129], 16, 2, seed=60)),
                    ("tiles", lc.attention_case([90, 40], [300, 40], 16, 2, seed=61)),
                    ("tiles split", lc.attention_case([40], [2000], 16, 2, seed=62)),
                    ("packed", lc.attention_case([70, 1], [70, 1], 8, 2, "TND", FP, seed=63)),
                    ("selected", lc.attention_case([1, 9], [3000, 700], 16, 2, k=6, seed=64))):
        d = to(c, dev)
        work.append((name, lambda d=d, **kw: list(call(d, **kw))))
    gen = torch.Generator().manual_seed(65)
    cu, T = lc.lengths([1, 30])
    kv = torch.tensor([200, 30], dtype=torch.int32).to(dev)
    table, pages = lc.table_for([200, 30], gen)
    cos, sin = (a.to(dev) for a in angles(256, 128))
    src = torch.randn(T, 5, 128, generator=gen).to(BF).to(dev)
    cu, table = cu.to(dev), table.to(dev)

    def append(**kw):
        dst = torch.zeros(pages, 128, 5, 128, dtype=BF, device=dev)
        rows = torch.zeros(T, 5, 64, dtype=torch.uint8, device=dev)
        scale = torch.zeros(T, 5, 4, dtype=torch.uint8, device=dev)
        m.msa_cache_append([m.CacheItem(src, dst, "BBND", rotate=True),
                            m.CacheItem(src, rows, "ROWS", scale, True)], cos, sin, table, cu, kv,
                           **kw)
        return [dst, rows, scale]

    work.append(("append", append))
    return work


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a, b))


def test_graph_replays(dev):
    """Each entry captured, with its outputs and workspace, and replayed three
    times with eager work between; two graphs' workspaces are their own."""
    for name, f in _entries(dev):
        log("graph", name)
        eager = f()
        torch.cuda.synchronize()
        graphs = []
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                out = f()
            graphs.append((g, out))
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for rep in range(3):
            for g, out in graphs:
                for o in out:
                    o.view(torch.uint8).fill_(0 if name == "append" else 255)
            f()
            torch.cuda.synchronize()
            for g, _ in graphs:
                g.replay()
            torch.cuda.synchronize()
            for _, out in graphs:
                assert same(out, eager), (name, rep)


def test_threads_on_streams(dev):
    work = _entries(dev)
    alone = [f() for _, f in work]
    streams = [torch.cuda.Stream(device=dev) for _ in work]
    torch.cuda.synchronize()
    got, errors = [[] for _ in work], []
    start = threading.Barrier(len(work))

    def go(i):
        try:
            start.wait()
            with torch.cuda.stream(streams[i]):
                for _ in range(4):
                    got[i].append(work[i][1]())
        except Exception as e:
            errors.append((work[i][0], repr(e)))

    threads = [threading.Thread(target=go, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i, (name, _) in enumerate(work):
        for x in got[i]:
            assert same(x, alone[i]), name


def test_keys_past_4_gib(dev):
    """Pages and packed keys on both sides of 4 GiB of the cache."""
    H = 8
    pages = (1 << 32) // (128 * H * 128 * 2) + 40
    k = torch.zeros(pages, 128, H, 128, dtype=BF, device=dev)
    v = torch.zeros(pages, 128, H, 128, dtype=BF, device=dev)
    c = lc.attention_case([1, 20], [1000, 700], 16, H, seed=70)
    far = torch.arange(c["k"].shape[0]) * 3 + pages - 3 * c["k"].shape[0]
    far[::2] = torch.arange(0, len(far), 2)
    k[far.to(dev)], v[far.to(dev)] = c["k"].to(dev), c["v"].to(dev)
    d = to(c, dev)
    near = call(d)
    d["k"], d["v"] = k, v
    d["table"] = torch.where(c["table"] >= 0, far[c["table"].clamp(min=0).long()].int(),
                             c["table"]).to(dev)
    assert int(d["table"].max()) * 128 * H * 128 * 2 > 1 << 32
    assert same(call(d), near)
    d["blocks"] = torch.tensor([0, 2, 3, 5], dtype=torch.int32, device=dev).expand(21, H, 4).contiguous()
    got = call(d)
    c["blocks"] = d["blocks"].cpu()
    check(c, *got)
    # the append, to the far pages
    import block_max_qk_amd as m
    src = torch.randn(21, H, 128, generator=torch.Generator().manual_seed(1)).to(BF).to(dev)
    m.msa_cache_append([m.CacheItem(src, k, "BBND")], None, None, d["table"], d["cu"], d["kv"])
    torch.cuda.synchronize()
    for t, b, pos in layer.positions(c["cu"], c["kv"], 21):
        assert torch.equal(k[int(d["table"][b, pos // 128]), pos % 128], src[t])
    # packed: a second request behind 4 GiB of the first's keys
    flat_k, flat_v = k.view(-1, H, 128), v.view(-1, H, 128)
    n = flat_k.shape[0]
    t = lc.attention_case([3, 50], [200, 300], 16, H, "TND", seed=71)
    flat_k[n - 300:], flat_v[n - 300:] = t["k"][200:].to(dev), t["v"][200:].to(dev)
    d = to(t, dev)
    near = call(d)
    q0 = torch.zeros_like(d["q"])
    q0[3:] = d["q"][3:]
    d["k"], d["v"] = flat_k, flat_v
    d["kv"] = torch.tensor([n - 300, 300], dtype=torch.int32, device=dev)
    got = call(d)
    torch.cuda.synchronize()
    t["kv"] = torch.tensor([200, 300], dtype=torch.int32)
    ref = layer.attention(t["q"], t["k"], t["v"], None, t["cu"], t["kv"], "TND", 3)
    tol_out, tol_lse = layer.attention_bounds(ref, BF)
    assert ((got[0].cpu().double() - ref.out).abs() <= tol_out)[3:].all()
    assert ((near[0].cpu().double() - ref.out).abs() <= tol_out)[3:].all()


def test_workspace_of_the_caller(dev):
    import block_max_qk_amd as m
    c = lc.attention_case([1, 1], [3000, 129], 16, 2, seed=72)
    d = to(c, dev)
    need = m.msa_attention_workspace(2, 2, 16, 2, c["table"].shape[1])
    ws = torch.full((need + 32,), 255, dtype=torch.uint8, device=dev)
    got = call(d, workspace=ws[:need])
    check(c, *got)
    assert (ws[need:] == 255).all()
    with pytest.raises(m.MsaError):
        call(d, workspace=ws[:need - 16])


@pytest.mark.parametrize("T,Hq,Hkv,k,steps", [
    # a decode loop's graph: slots fill and empty, one request runs far ahead
    (8, 16, 2, 0, [([1] * 8, [100] * 8), ([1] * 5 + [0] * 3, [4000, 1, 0, 129, 128, 0, 7, 300]),
                   ([2, 0, 3, 0, 0, 1, 0, 0], [5000, 9, 3, 1, 0, 1025, 0, 0])]),
    # chunks of changing shares of the same rows
    (200, 16, 2, 0, [([100, 100], [100, 100]), ([190, 1], [2900, 2900]), ([0, 150], [5, 150])]),
    (8, 16, 2, 4, [([1] * 8, [900] * 8), ([3, 1] + [0] * 6, [4000, 1] + [0] * 6)]),
    (300, 16, 4, 4, [([150, 150], [600, 150]), ([299, 0], [3000, 40]), ([1, 100], [2000, 2000])]),
])
def test_graph_with_new_lengths(T, Hq, Hkv, k, steps, dev):
    """One captured call, replayed as the lengths in its tensors change: the
    split follows them, within the launch that was captured."""
    B, width = len(steps[0][0]), 40
    gen = torch.Generator().manual_seed(90 + T)
    c = lc.attention_case([0] * B, [128 * width] * B, Hq, Hkv, T_extra=T, k=k, seed=91)
    d = to(c, dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out, lse = call(d)
    torch.cuda.current_stream().wait_stream(s)
    for q_lens, kv_lens in steps + steps[:1]:
        cu, _ = lc.lengths(q_lens, T - sum(q_lens), 0)
        kv = torch.tensor(kv_lens, dtype=torch.int32)
        c["q"] = torch.randn(T, Hq, 128, generator=gen).to(BF)
        c["cu"], c["kv"] = cu, kv
        for n in ("q", "cu", "kv"):
            d[n].copy_(c[n])
        g.replay()
        torch.cuda.synchronize()
        n = int(cu[-1])
        check(c, out, lse)
        assert torch.isnan(out[n:]).all() and torch.isnan(lse[n:]).all()
