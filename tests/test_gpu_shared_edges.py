"""Shared prefixes where their parts meet odd bounds: shares of own keys that hold none,
small values, scales at their ends, positions and lengths near the ends of int32."""
import pytest
import torch

import gqa_attention_kv_gb300 as gq
from test_gpu_shared import DEV, Case, one_group

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,n,H,D", [("bf16", 60, 1, 128), ("bf16", 200, 4, 64),
                                       ("int8", 120, 2, 64), ("e4m3", 37, 8, 128)])
def test_shares_that_lie_in_gaps(fmt, n, H, D):
    """Own keys of 1 to 20: a share of four chunks of 34 a unit holds keys in one of eight, and
    the others follow one another without work between them."""
    c = Case(fmt, gq.LINEAR, one_group(n, 48), [1 + (7 * i) % 20 for i in range(n)], 1, 2 * H, H, D,
             16, n + D)
    want = c.check()
    need = gq.attn_decode_shared_workspace_size(c.cache, n, 1, 2 * H, c.longest, c.max_prefix)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    for _ in range(50):
        assert torch.equal(c.run(workspace=ws), want)
