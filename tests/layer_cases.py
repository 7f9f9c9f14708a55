"""Small seeded inputs for the cache append and the attention tests."""
import torch

P, D = 128, 128


def lengths(q_lens, T_extra=0, first=0):
    cu = [first]
    for n in q_lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32), cu[-1] + T_extra


def table_for(kv_lens, gen, spare=2, width=None, tail=-1):
    """(block_table [B, width], pages): scattered pages, `tail` behind each
    request's last block."""
    nb = [-(-max(n, 0) // P) for n in kv_lens]
    pages = sum(nb) + spare
    perm = torch.randperm(pages, generator=gen)
    table = torch.full((len(nb), width or max(max(nb), 1)), tail, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nb):
        table[b, :n] = perm[at:at + n].int()
        at += n
    return table, pages


def cache_shape(layout, pages, H, last=D):
    return (pages, P, H, last) if layout == "BBND" else (pages, H, P, last)


def attention_case(q_lens, kv_lens, Hq, Hkv, layout="BBND", dtype=torch.bfloat16, mode=3, seed=0,
                   T_extra=0, first=0, width=None, k=0, tail=-1):
    gen = torch.Generator().manual_seed(1000 + seed)
    cu, T = lengths(q_lens, T_extra, first)
    c = {"cu": cu, "kv": torch.tensor(kv_lens, dtype=torch.int32), "layout": layout, "mode": mode,
         "table": None, "blocks": None}

    def normal(*shape):
        return torch.randn(shape, generator=gen).to(dtype)

    c["q"] = normal(T, Hq, D)
    if layout == "TND":
        n = sum(max(x, 0) for x in kv_lens)
        c["k"], c["v"] = normal(n, Hkv, D), normal(n, Hkv, D)
    else:
        c["table"], pages = table_for(kv_lens, gen, width=width, tail=tail)
        c["k"] = normal(*cache_shape(layout, pages, Hkv))
        c["v"] = normal(*cache_shape(layout, pages, Hkv))
    if k:
        nb = max(-(-max(kv_lens) // P), 1)
        picks = torch.rand(T, Hkv, nb, generator=gen).argsort(-1)[..., :k]
        c["blocks"] = torch.full((T, Hkv, k), -1, dtype=torch.int32)
        c["blocks"][..., :picks.shape[-1]] = picks.sort(-1).values.int()
    return c
