"""Attention cases of the 256-row tiles, by name: what makes the sizes choose
them, and whether the tiles are split over the keys.

name: (q_lens, kv_lens, Hq, Hkv, layout, table width or None, split)"""

CASES = {
    "one prompt, whole": ([1000], [1000], 64, 8, "BBND", None, False),
    "one chunk, split evenly": ([520], [6000], 64, 8, "BBND", None, True),
    "a wide table, split by length": ([515, 301], [515, 430], 64, 8, "BBND", 16, True),
    "parts of both requests": ([515, 301], [5000, 3000], 64, 8, "BNBD", None, True),
    "parts of one request": ([330, 330, 240], [330, 9000, 2000], 64, 8, "BBND", None, True),
    "packed prompts": ([700, 1, 0, 499], [700, 1, 30, 499], 64, 8, "TND", None, False),
    "packed keys, split": ([600, 500], [2600, 500], 64, 8, "TND", None, True),
    "a group of more than a tile": ([70], [2048], 600, 2, "BBND", None, False),
    "a group that does not divide the tile": ([900, 700], [1400, 701], 40, 8, "BNBD", 16, True),
    "one head a group": ([4500], [4500], 8, 8, "BBND", None, True),
    "heads of their own, packed": ([4400, 3900], [4400, 3900], 8, 8, "TND", None, True),
}


def sizes(name):
    """Arguments of the plan's queries: T, B, Hq, Hkv, max_blocks."""
    q_lens, kv_lens, Hq, Hkv, layout, width, _ = CASES[name]
    if layout == "TND":
        mb = (sum(kv_lens) + 127) // 128
    else:
        mb = width or max(-(-n // 128) for n in kv_lens)
    return sum(q_lens), len(q_lens), Hq, Hkv, mb
