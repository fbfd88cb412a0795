"""Calls at the ends of what the latent operators take, without a GPU."""

import paged_kv_cache_111_gb300 as pkv
from test_latent_host import OK, latent_attn, lib  # noqa: F401  (lib: the fixture)


def test_the_workspace_of_an_empty_batch_is_that_of_any(lib):  # noqa: F811
    need = pkv.latent_paged_attn_workspace_size(2, 2, 1, 64, 16)
    assert pkv.latent_paged_attn_workspace_size(0, 0, 0, 0, 16) == need
    assert latent_attn(lib, S=0, T=0) == (OK, need)
