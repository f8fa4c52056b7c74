"""What the prompt's calls keep on the host: the sizes of some workspaces, not of
every number of rows there ever was."""
import gc

import sparse_attention_top_gb300 as gb


def test_sizes_of_packed_prompts_are_not_kept_for_good():
    sizes = gb.prefill._prompt_bytes
    sizes(1, 1, 8, 2, 64)
    gc.collect()
    before = len(gc.get_objects())
    for rows in range(1, 20001):
        assert sizes(rows, rows % 7 + 1, 8, 2, 64) > 0
    gc.collect()
    assert sizes.cache_info().currsize <= 1024
    assert len(gc.get_objects()) - before < 5000
    assert sizes(20000, 3, 8, 2, 64) == gb.gbtopk_prompt_workspace_bytes(20000, 3, 8, 2, 64)
