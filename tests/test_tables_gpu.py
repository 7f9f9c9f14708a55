"""The step's tables against the oracle (oracle/layer.py), every figure equal:
lengths of zero and one, blocks that the tokens just fill or begin, rows out of
order and out of range, free lists that are short, padded steps, batches past one
group of requests, the count updated in place, graphs, streams, and the steps
that follow with the tables."""
import random
import sys

import pytest
import torch

from oracle import layer

pytestmark = pytest.mark.gpu
P = 128


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_max_qk_amd
    block_max_qk_amd.load_library()
    return torch.device("cuda:0")


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def case(new, ctx, MB, R=None, rows="mixed", spare=5, pad=0, width=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    B = len(new)
    R = B + 3 if R is None else R
    width = MB if width is None else width
    held = [min(MB, -(-max(c, 0) // P)) for c in ctx]
    need = sum(min(MB, -(-(max(c, 0) + max(n, 0)) // P)) - h for n, c, h in zip(new, ctx, held))
    free = max(0, need + spare)
    pages = torch.randperm(sum(held) + free, generator=gen).int()
    pool = torch.full((R, width), -7, dtype=torch.int32)    # (stale entries: never read)
    order = torch.randperm(R, generator=gen)[:B].int() if rows == "mixed" else rows
    for b, h in enumerate(held):
        r = b if order is None else int(order[b])
        if 0 <= r < R:
            pool[r, :h] = pages[sum(held[:b]):sum(held[:b + 1])]
    free_pages = torch.full((free + 4,), -5, dtype=torch.int32)
    free_pages[:free] = pages[sum(held):]
    return {"new": i32(new), "ctx": i32(ctx), "rows": order, "pool": pool, "free": free_pages,
            "count": i32([free, 99]), "MB": MB, "T": sum(max(n, 0) for n in new) + pad}


def expect(c):
    return layer.step_tables(c["new"], c["ctx"], c["rows"], c["pool"], c["free"],
                             int(c["count"][0]), c["MB"], c["T"])


def call(c, dev, in_place=False, **kw):
    import block_max_qk_amd as m
    d = {n: (x.to(dev) if torch.is_tensor(x) else x) for n, x in c.items()}
    out = m.new_step_tables(len(c["new"]), c["T"], c["MB"], dev)
    for t in out:
        t.fill_(-99)
    left = d["count"] if in_place else torch.full((2,), -99, dtype=torch.int32, device=dev)
    m.msa_step_tables(d["new"], d["ctx"], d["pool"], d["free"], d["count"], out, rows=d["rows"],
                      free_out=None if in_place else left, **kw)
    torch.cuda.synchronize()
    if not in_place:
        assert torch.equal(d["count"].cpu(), c["count"])
    return {**out._asdict(), "free": left, "pool": d["pool"]}


def same(got, want):
    for n, w in want.items():
        w = w if torch.is_tensor(w) else torch.tensor(w, dtype=torch.int64)
        assert torch.equal(got[n].cpu().long(), w.long()), n


def run(c, dev, **kw):
    same(call(c, dev, **kw), expect(c))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("new,ctx,MB", [
    ([1], [0], 1), ([0], [0], 1), ([0, 0], [5, 0], 3), ([128], [0], 2), ([1], [128], 2),
    ([1], [127], 2), ([129, 1, 0, 256], [127, 1, 300, 0], 5), ([1000], [1], 9),
    ([300, 1], [200, 640], 4),                     # tokens past the last block
    ([1, 1], [5000, 512], 4),                      # so are these, and their context
    ([-3, 2], [4, -9], 2),                         # negative lengths count as none
])
def test_lengths(new, ctx, MB, in_place, dev):
    log("lengths", new, ctx, MB, in_place)
    run(case(new, ctx, MB), dev, in_place=in_place)


def test_no_requests(dev):
    run(case([], [], 3, R=2, pad=0), dev)
    run(case([], [], 3, R=0, pad=700), dev, in_place=True)


@pytest.mark.parametrize("rows", [None, i32([2, -1, 0, 9]), i32([3, 2, 1, 0])])
def test_rows(rows, dev):
    """Rows out of order; a row that is none holds no pages and takes none."""
    run(case([200, 130, 1, 700], [100, 300, 128, 0], 7, R=4, rows=rows), dev)


@pytest.mark.parametrize("spare", [-1, -4, -100, 0])
@pytest.mark.parametrize("in_place", [False, True])
def test_free_list_runs_out(spare, in_place, dev):
    run(case([300, 2, 129, 500], [0, 127, 255, 3], 8, spare=spare), dev, in_place=in_place)


def test_count_past_the_list(dev):
    c = case([300, 2], [0, 127], 8)
    c["free"] = c["free"][:2].contiguous()
    c["count"] = i32([1000, 0])
    run(c, dev)
    c["count"] = i32([-4, 0])
    run(c, dev)


@pytest.mark.parametrize("B", [2, 65, 300, 511, 513, 1500])
@pytest.mark.parametrize("pad,in_place", [(0, True), (777, False)])
def test_batches(B, pad, in_place, dev):
    log("batch", B, pad)
    rng = random.Random(B)
    new = [rng.choice([0, 1, 1, 1, 5, 200]) for _ in range(B)]
    ctx = [rng.randint(0, 2000) for _ in range(B)]
    run(case(new, ctx, 20, pad=pad, width=23, spare=rng.choice([-3, 9]), seed=B), dev,
        in_place=in_place)


def test_groups_of_64(dev):
    """More requests than 512 groups of 64."""
    B = 33000
    rng = random.Random(3)
    run(case([rng.choice([0, 1, 3]) for _ in range(B)], [rng.randint(0, 500) for _ in range(B)], 5,
             rows=None), dev)


def test_the_most_requests(dev):
    """2^20 requests, all but a few of them empty, and large page numbers."""
    import block_max_qk_amd as m
    B, T = 1 << 20, 1000
    gen = torch.Generator().manual_seed(5)
    at = torch.randperm(B, generator=gen)[:500].sort().values
    new, ctx = torch.zeros(2, B, dtype=torch.int32)
    new[at], ctx[at] = 2, 127
    pool = torch.full((B, 2), 1 << 28, dtype=torch.int32)
    free = (torch.randperm(600, generator=gen) + (1 << 30)).int()
    d = [x.to(dev) for x in (new, ctx, pool, free, i32([600, 0]))]
    out = m.new_step_tables(B, T, 2, dev)
    m.msa_step_tables(*d, out)
    torch.cuda.synchronize()
    cu = torch.zeros(B + 1, dtype=torch.long)
    cu[1:] = new.long().cumsum(0)
    pages = free.flip(0)[:500].long()
    assert torch.equal(out.cu_seqlens_q.cpu().long(), cu)
    assert torch.equal(out.cu_pages.cpu().long(), cu // 2)
    assert torch.equal(out.kv_len.cpu(), new + ctx) and not out.start_loc.any()
    table = torch.full((B, 2), -1, dtype=torch.int32)
    table[at, 0], table[at, 1] = 1 << 28, pages.int()
    assert torch.equal(out.block_table.cpu(), table)
    pool[at, 1] = pages.int()
    assert torch.equal(d[2].cpu(), pool) and d[4].tolist() == [100, 0]
    slots = torch.stack([torch.full((500,), (1 << 35) + 127), pages * P], 1).flatten()
    assert torch.equal(out.slots.cpu(), slots)
    assert torch.equal(out.positions.cpu().view(500, 2), i32([[127, 128]]).expand(500, 2))


def test_long_prompt(dev):
    """One request's blocks and tokens shared by many workgroups."""
    run(case([70001], [130], 700, pad=100), dev)
    run(case([20000, 1, 3000], [0, 70000, 12], 600), dev)


def test_more_tokens_than_rows(dev):
    """The sum past T: nothing is written past the tensors, and the prefix sums
    end at T."""
    c = case([100, 50, 60], [0, 3, 9], 2)
    c["T"] = 120
    got = call(c, dev)
    assert got["cu_seqlens_q"].tolist() == [0, 100, 120, 120]
    want = expect({**c, "T": 210})
    assert got["positions"].tolist() == want["positions"][:120]
    assert got["slots"].tolist() == want["slots"][:120]
    same({n: got[n] for n in ("kv_len", "block_table", "pool", "free")},
         {n: want[n] for n in ("kv_len", "block_table", "pool", "free")})


def test_allocating_form_and_streams(dev):
    import block_max_qk_amd as m
    c = case([3, 400, 1], [0, 100, 128], 6, pad=5)
    d = {n: (x.to(dev) if torch.is_tensor(x) else x) for n, x in c.items()}
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    out = m.step_tables(d["new"], d["ctx"], d["pool"], d["free"], d["count"], c["T"],
                        rows=d["rows"], stream=side)
    torch.cuda.current_stream(dev).wait_stream(side)
    torch.cuda.synchronize()
    same({**out._asdict(), "pool": d["pool"], "free": d["count"]}, expect(c))
    # a narrower bound than the pool's width
    c["MB"] = 2
    d = {n: (x.to(dev) if torch.is_tensor(x) else x) for n, x in c.items()}
    out = m.step_tables(d["new"], d["ctx"], d["pool"], d["free"], d["count"], c["T"],
                        rows=d["rows"], max_blocks=2)
    same({**out._asdict(), "pool": d["pool"], "free": d["count"]}, expect(c))


def test_captured_and_replayed(dev):
    """A decode step captured once: each replay takes its pages where the last
    one left the list, in place, with the lengths that it is given."""
    import block_max_qk_amd as m
    c = case([1, 1, 1, 1], [126, 3, 255, 0], 9, spare=20, pad=300)
    d = {n: (x.to(dev) if torch.is_tensor(x) else x) for n, x in c.items()}
    out = m.new_step_tables(4, c["T"], 9, dev)

    def step():
        m.msa_step_tables(d["new"], d["ctx"], d["pool"], d["free"], d["count"], out,
                          rows=d["rows"])

    before = {n: d[n].clone() for n in ("pool", "count")}
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream(dev).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n, x in before.items():
        d[n].copy_(x)
    for new in ([2, 200, 1, 1], [1, 0, 130, 1], [1, 1, 1, 1], [0, 0, 0, 299], [1, 1, 1, 1]):
        graph.replay()
        torch.cuda.synchronize()
        want = expect(c)
        same({**out._asdict(), "pool": d["pool"], "free": d["count"]}, want)
        c["pool"], c["count"] = want["pool"], i32(want["free"])
        c["ctx"], c["new"] = i32(want["kv_len"]), i32(new)
        d["ctx"].copy_(c["ctx"])
        d["new"].copy_(c["new"])


def test_refusals(dev):
    import block_max_qk_amd as m
    c = case([3, 4], [0, 100], 6)
    d = {n: (x.to(dev) if torch.is_tensor(x) else x) for n, x in c.items()}
    out = m.new_step_tables(2, c["T"], 6, dev)

    def go(out=out, **kw):
        a = {**d, **kw}
        return m.msa_step_tables(a["new"], a["ctx"], a["pool"], a["free"], a["count"], out,
                                 rows=a["rows"], free_out=a.get("left"))

    for bad in (dict(new=d["new"].long()), dict(ctx=d["ctx"][:1]), dict(pool=d["pool"][0]),
                dict(pool=d["pool"].cpu()), dict(rows=d["rows"][:1]), dict(count=d["count"][:1]),
                dict(left=d["count"][:1]), dict(free=d["free"][None]),
                dict(pool=d["pool"].t()), dict(new=d["new"].cpu(), ctx=d["ctx"].cpu()),
                dict(out=out._replace(slots=out.slots.int())),
                dict(out=out._replace(cu_pages=out.cu_pages[:2])),
                dict(out=out._replace(positions=out.positions[:2]))):
        with pytest.raises(ValueError):
            go(**bad)
    for bad in (dict(out=out._replace(kv_len=d["ctx"])),              # written over its input
                dict(out=out._replace(start_loc=out.kv_len)),
                dict(left=out.cu_pages[:2]), dict(free=out.positions),
                dict(pool=d["pool"][:, :4].contiguous())):           # narrower than the table
        with pytest.raises(m.MsaError):
            go(**bad)
