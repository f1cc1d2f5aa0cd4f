"""What the 8-bit cache, attention weights and eviction refuse, each refusal by its own reason, without
a GPU.  Nothing here launches."""

import pytest

from paged_kv_cache_exact_b200 import binding as B
from test_cache_cpu import ATTN, ATTN_OK, W_TAIL, _call

MOST = 65535 * 128                          # keys of a prompt's weights: a grid's second axis of 128-key tiles


@pytest.mark.parametrize("kw", [dict(q_len=300), dict(q_len=2, S=40)], ids=["rows", "scores too many for the split kernel"])
def test_a_prompts_weights_over_too_many_keys_are_refused_before_the_attention_runs(kw):
    kw = dict(kw, max_len=MOST + 1, stride=MOST + 1, maxp=1 << 20)
    assert _call("paged_attn_weights", ATTN + W_TAIL[0], ATTN_OK + W_TAIL[1], kw) == B.PKV_ERR_UNSUPPORTED
    # one key fewer is not refused for its size: the workspace is asked for
    kw.update(max_len=MOST, stride=MOST, ws=None)
    assert _call("paged_attn_weights", ATTN + W_TAIL[0], ATTN_OK + W_TAIL[1], kw) == B.PKV_ERR_WORKSPACE
