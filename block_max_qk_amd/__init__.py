"""MSA index-branch block scores on AMD Instinct MI355X (gfx950).

The operator lives in the HIP library ``libmsa_index_score.so`` (C ABI in
``include/msa_index_score.h``), with the top-k block selection over its
output (``msa_block_topk``), the cache append in front of it
(``msa_cache_append``, by several position axes ``msa_cache_append_axes``), the
attention behind it (``msa_attention``, ``msa_block_attention``, with capped,
biased or narrowed scores ``msa_attention_ex``) and the tables of a serving step
(``msa_step_tables``); this package holds its sources (``csrc/``), the
hipcc build step (``build.py``) and a ctypes binding with the same names.
"""
from ._binding import (  # noqa: F401
    EXPORTED,
    LIB_PATH,
    CacheItem,
    MsaError,
    MsaLayoutError,
    MsaTensor,
    StepTables,
    attention,
    block_attention,
    block_topk,
    describe,
    index_score,
    load_library,
    msa_attention,
    msa_attention_ex_workspace,
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
    msa_step_tables,
    new_step_tables,
    step_tables,
)
