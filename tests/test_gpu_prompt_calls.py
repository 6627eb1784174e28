"""What a program meets around the prompt chunk's calls: the status of calls without rows.  References and
tolerances are those of test_gpu_prompt.py."""
import pytest
import torch

import gated_delta_rule_16_gb300 as gdn
from test_gpu_prompt import KINDS, Case, _built, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("used", [False, True])
def test_status_after_a_call_without_rows(kind, used):
    c = Case([(30, 20)], kind=kind)
    ws = gdn.Workspace()
    if used:
        c.call(workspace=ws)
    else:
        ws.buf = torch.empty(1 << 26, dtype=torch.uint8, device=c.q.device)
    for q, table, lens, cu in ((c.q[:0], c.table, c.lens, i32([0, 0])), (c.q[:0], c.table[:0], c.lens[:0], i32([0])),
                               (c.q, c.table[:0], c.lens[:0], i32([0]))):
        ws.buf.fill_(0xFF)  # what memory held before, or an earlier call's status
        gdn.gdn_paged_prefill(q, c.k, c.v, table, lens, cu, workspace=ws, **c.scales)
        assert gdn.gdn_paged_prefill_status(ws) == 0
        assert (ws.buf[4:] == 0xFF).all()
    c.check(workspace=ws)
    assert gdn.gdn_paged_prefill_status(ws) == 0
