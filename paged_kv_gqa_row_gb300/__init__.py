"""GB300 (sm_103a) paged decode / step attention.

The product is the C-ABI library ``liblnk.so`` (declared in ``include/lnk.h``);
this package holds its CUDA sources (``csrc/``), the build step (``build.py``)
and a thin ctypes binding with the C names (``binding.py``).
"""
from .binding import (  # noqa: F401
    DEV_TIMEOUT,
    EXPORTED,
    KV_BF16,
    KV_E2M1,
    KV_E4M3,
    LIBRARY_PATH,
    AttnDesc,
    LatentDesc,
    LnkError,
    Pager,
    RopeDesc,
    attn_desc,
    latent_desc,
    lnk_latent_append,
    lnk_latent_copy_pages,
    lnk_latent_decode_attn,
    lnk_latent_prompt_attn,
    lnk_latent_step_attn,
    lnk_latent_workspace_size,
    lnk_paged_append_rope,
    lnk_paged_copy_pages,
    lnk_paged_copy_pages_layers,
    lnk_paged_decode_attn,
    lnk_paged_decode_step,
    lnk_paged_decode_step_launches,
    lnk_paged_decode_attn_static,
    lnk_paged_page_bytes,
    lnk_paged_read_tokens,
    lnk_paged_step_attn,
    lnk_paged_workspace_size,
    lnk_rope_inv_freq,
    lnk_selftest_wait_timeout,
    lnk_status_string,
    rope_desc,
)
