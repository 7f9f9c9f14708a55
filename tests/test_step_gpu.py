"""A serving step as a server runs it: the step's tables, the append with position
axes into the pages that they hand out, and attention with images that see
themselves, a cap and a bias, over chunks and decode steps; against the oracle step
by step, and captured whole into a graph whose replays follow the requests."""
import sys

import pytest
import torch

from oracle import layer

pytestmark = pytest.mark.gpu
P, D = 128, 128
HQ, HKV, ROT, AXES = 8, 2, 64, 3
PAIRS = [r % AXES for r in range(ROT // 2)]


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_max_qk_amd
    block_max_qk_amd.load_library()
    return torch.device("cuda:0")


def angles(n):
    inv = 10000.0 ** (-torch.arange(0, ROT, 2, dtype=torch.float64) / ROT)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def axis_of(pos):
    """Time, height and width of a token: rows of 7 behind the first 20 tokens."""
    image = pos >= 20
    return torch.stack([torch.where(image, 20, pos), torch.where(image, 20 + (pos - 20) // 7, pos),
                        torch.where(image, 20 + (pos - 20) % 7, pos)]).int()


def visible_of(pos, kv):
    """Images are tokens 50 to 189 of a sequence, in two of 70: a token of one sees
    to its end, as far as it is there."""
    image = (pos >= 50) & (pos < 190)
    end = torch.where(image, 50 + ((pos - 50) // 70 + 1) * 70, pos + 1)
    return torch.stack([torch.zeros_like(pos), torch.minimum(torch.maximum(end, pos + 1), kv)],
                       1).int()


class Server:
    def __init__(self, dev, R=5, MB=4, pages=14):
        self.pool = torch.full((R, MB), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(pages, dtype=torch.int32, device=dev).flip(0).contiguous()
        self.count = torch.tensor([pages, 0], dtype=torch.int32, device=dev)
        self.k = torch.zeros(pages, P, HKV, D, dtype=torch.bfloat16, device=dev)
        self.v = torch.zeros_like(self.k)
        self.cos, self.sin = (x.to(dev) for x in angles(300))
        self.slopes = torch.tensor([2.0 ** (-i - 1) for i in range(HQ)], device=dev)

    def step(self, new, ctx, rows, qkv, out=None):
        """One step on device tensors, all of it asynchronous."""
        import block_max_qk_amd as m
        T = qkv.shape[0]
        t = m.step_tables(new, ctx, self.pool, self.free, self.count, T, rows=rows)
        pos = t.positions
        q = torch.empty(T, HQ, D, dtype=qkv.dtype, device=qkv.device)
        m.msa_cache_append(
            [m.CacheItem(qkv[:, :HQ], q, "ROWS", rotate=True),
             m.CacheItem(qkv[:, HQ:HQ + HKV], self.k, "BBND", rotate=True),
             m.CacheItem(qkv[:, HQ + HKV:], self.v, "BBND")],
            self.cos, self.sin, t.block_table, t.cu_seqlens_q, t.kv_len,
            axis_positions=axis_of(pos), pair_axes=PAIRS)
        b = torch.searchsorted(t.cu_seqlens_q[1:], torch.arange(T, device=qkv.device,
                                                                dtype=torch.int32), right=True)
        kv = torch.cat([t.kv_len, t.kv_len.new_zeros(1)])[b]
        vis = visible_of(pos, kv)
        o, lse = m.attention(q, self.k, self.v, t.block_table, t.cu_seqlens_q, t.kv_len, "BBND",
                             sparse_mode=0, softcap=25.0, slopes=self.slopes, visible=vis,
                             return_lse=True)
        return t, q, vis, o, lse

    def clone(self):
        s = object.__new__(Server)
        s.__dict__ = {n: x.clone() for n, x in self.__dict__.items()}
        return s


def rotated(x, pos):
    """Rows [n, H, D] rotated in binary64 by the axes of their positions."""
    cos, sin = (a.double() for a in angles(300))
    at = axis_of(pos).long()[PAIRS].T                       # [n, pairs]
    r = torch.arange(ROT // 2)
    c, s = cos[at, r][:, None], sin[at, r][:, None]
    x = x.double()
    a, b = x[..., :ROT // 2], x[..., ROT // 2:ROT]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., ROT:]], -1)


def test_chunks_and_decode(dev):
    """Three requests join and leave: chunks, single tokens, one that brings
    nothing, a padded step."""
    gen = torch.Generator().manual_seed(9)
    srv = Server(dev)
    ctx = {0: 0, 3: 0, 1: 0}
    told = {r: ([], []) for r in ctx}                       # rotated keys, values by row
    steps = [([(0, 130)], 130), ([(0, 60), (3, 35)], 95), ([(3, 100), (1, 1), (0, 1)], 110),
             ([(0, 1), (1, 1), (3, 1)], 3), ([(1, 200), (0, 0), (3, 2)], 207)]
    for n, (brings, T) in enumerate(steps):
        log("step", n, brings)
        rows = [r for r, _ in brings]
        new = [q for _, q in brings]
        qkv = torch.randn(T, HQ + 2 * HKV, D, generator=gen).to(torch.bfloat16)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        want = layer.step_tables(new, [ctx[r] for r in rows], rows, srv.pool.cpu(),
                                 srv.free.cpu(), int(srv.count[0]), 4, T)
        t, q, vis, o, lse = srv.step(i32(new), i32([ctx[r] for r in rows]), i32(rows),
                                     qkv.to(dev))
        torch.cuda.synchronize()
        for name, x in t._asdict().items():
            w = want[name] if torch.is_tensor(want[name]) else torch.tensor(want[name])
            assert torch.equal(x.cpu().long(), w.long()), name
        assert torch.equal(srv.pool.cpu(), want["pool"]) and srv.count.tolist() == want["free"]
        # the pages hold every request's rotated keys and its values, old and new
        pos = torch.tensor(want["positions"])
        at = 0
        for r, k in brings:
            told[r][0].append(rotated(qkv[at:at + k, HQ:HQ + HKV], pos[at:at + k]))
            told[r][1].append(qkv[at:at + k, HQ + HKV:])
            ctx[r] += k
            at += k
            keys, vals = torch.cat(told[r][0]), torch.cat(told[r][1])
            j = torch.arange(ctx[r])
            page = want["pool"][r, j // P].long()
            got = srv.k.cpu()[page, j % P].double()
            # half a step of bf16, and three float32 roundings of terms below 8
            assert ((got - keys).abs() <= keys.abs() * 2.0 ** -8 + 3 * 8 * 2.0 ** -24 + 1e-30).all()
            assert torch.equal(srv.v.cpu()[page, j % P], vals)
        used = sum(new)
        gotq = q.cpu()[:used].double()
        wantq = rotated(qkv[:used, :HQ], pos[:used])
        assert ((gotq - wantq).abs() <= wantq.abs() * 2.0 ** -8 + 3 * 8 * 2.0 ** -24).all()
        ref = layer.attention_forms(q.cpu(), srv.k.cpu(), srv.v.cpu(), t.block_table.cpu(),
                                    t.cu_seqlens_q.cpu(), t.kv_len.cpu(), "BBND", 0, None, 25.0,
                                    srv.slopes.cpu(), vis.cpu())
        tol, tol_lse = layer.forms_bounds(ref, torch.bfloat16)
        assert ((o.cpu().double() - ref.out).abs() <= tol)[:used].all()
        assert ((lse.cpu().double() - ref.lse).abs() <= tol_lse)[:used].all()
        assert (ref.keys[:used] > 0).all()


def test_the_whole_step_captured(dev):
    """One graph of tables, append and attention, replayed over decode steps whose
    lengths the tables carry on, with the eager step on a copy beside it."""
    gen = torch.Generator().manual_seed(10)
    srv = Server(dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    rows = i32([2, 0, 4])
    first = torch.randn(300, HQ + 2 * HKV, D, generator=gen).to(torch.bfloat16).to(dev)
    srv.step(i32([126, 60, 40]), i32([0, 0, 0]), rows, first)
    new, ctx = i32([1, 1, 1]), i32([126, 60, 40])
    qkv = torch.zeros(4, HQ + 2 * HKV, D, dtype=torch.bfloat16, device=dev)
    twin = srv.clone()
    before = srv.clone()
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        srv.step(new, ctx, rows, qkv)
    torch.cuda.current_stream(dev).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t, _, _, o, lse = srv.step(new, ctx, rows, qkv)
        ctx.copy_(t.kv_len)
    ctx.copy_(i32([126, 60, 40]))
    for n in ("pool", "count", "k", "v"):
        getattr(srv, n).copy_(getattr(before, n))
    length = i32([126, 60, 40])
    for _ in range(5):
        qkv.copy_(torch.randn(qkv.shape, generator=gen))
        graph.replay()
        et, _, _, eo, else_ = twin.step(new, length, rows, qkv)
        torch.cuda.synchronize()
        length = et.kv_len
        assert torch.equal(t.block_table, et.block_table) and torch.equal(t.slots, et.slots)
        assert torch.equal(srv.pool, twin.pool) and torch.equal(srv.count, twin.count)
        assert torch.equal(srv.k, twin.k) and torch.equal(srv.v, twin.v)
        assert torch.equal(o[:3], eo[:3]) and torch.equal(lse[:3], else_[:3])
    assert length.tolist() == [131, 65, 45] and int((srv.pool[2] >= 0).sum()) == 2
