"""MSA index-branch block scores on AMD Instinct MI355X (gfx950).

The operator lives in the HIP library ``libmsa_index_score.so`` (C ABI in
``include/msa_index_score.h``), with the top-k block selection over its
output (``msa_block_topk``), the cache append in front of it
(``msa_cache_append``) and the attention behind it (``msa_attention``,
``msa_block_attention``); this package holds its sources (``csrc/``), the
hipcc build step (``build.py``) and a ctypes binding with the same names.
"""
from ._binding import (  # noqa: F401
    EXPORTED,
    LIB_PATH,
    CacheItem,
    MsaError,
    MsaLayoutError,
    MsaTensor,
    attention,
    block_attention,
    block_topk,
    describe,
    index_score,
    load_library,
    msa_attention,
    msa_attention_tile_rows,
    msa_attention_workspace,
    msa_block_attention,
    msa_block_topk,
    msa_cache_append,
    msa_index_score,
    msa_index_score_kernel_family,
    msa_index_score_mxfp4,
    msa_index_score_out_width,
    msa_status_str,
)
