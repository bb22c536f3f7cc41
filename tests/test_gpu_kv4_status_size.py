"""A status tensor is two numbers: fewer are refused before anything is launched."""
import pytest
import torch

import expert_routing_moe_gb300 as moe
from _gpu import DEV

pytestmark = pytest.mark.gpu


def test_a_short_status_is_refused():
    i32 = dict(dtype=torch.int32, device=DEV)
    pages = moe.KvPages(1, 4, 1, 64, 1, 128, DEV)
    cache, starts = pages.layer(0), torch.tensor([0, 1], **i32)
    pages.reserve(torch.ones(1, **i32))
    short = torch.zeros(1, **i32)
    x = torch.randn(1, 3 * 64, device=DEV).bfloat16()
    q, out = torch.empty(1, 1, 64, dtype=torch.bfloat16, device=DEV), torch.empty(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(moe.attention_kv4_workspace(1, 1, 1, 64), dtype=torch.uint8, device=DEV)
    for stream in (None, torch.cuda.current_stream()):
        for call in (lambda: moe.moe_qk_norm_rope(x, 1, 1, q, cache=cache, q_start=starts, st=short, stream=stream),
                     lambda: moe.moe_kv4_read(cache, starts, out, None, st=short, stream=stream),
                     lambda: moe.moe_attention_kv4(q, cache, starts, out, 0.1, max_new=1, workspace=ws, st=short, stream=stream),
                     lambda: moe.moe_kv4_reserve(pages.pool, short, pages.workspace, st=short, stream=stream),
                     lambda: moe.moe_kv4_assign(pages.pool, short, st=short, stream=stream),
                     lambda: moe.moe_kv4_compact(pages.pool, None, pages.workspace, st=short, stream=stream)):
            with pytest.raises(moe.MoeError, match="status"):
                call()
