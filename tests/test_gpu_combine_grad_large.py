"""Combine's gradient for so many tokens that one grid of a workgroup a token would
pass 2^32 threads."""
import pytest
import torch

from combine_ep_get_layout_amd import ep
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [ep.MODE_NORMAL, ep.MODE_RANK_MAJOR])
@pytest.mark.parametrize("T", [(1 << 24) + 5, 1 << 23, (1 << 23) + 1])
def test_tokens_past_a_grid(T, mode):
    """One expert, top-1, eight channels, every seventh token without a row.  Compared exactly:
    weights are powers of two and values small integers, so each product and each sum of
    eight of them is exact in bf16 and fp32."""
    say("combine_backward", T, mode)
    H = 8
    p = ep.Problem(1, T, H, 1, 1, mode=mode)
    t = torch.arange(T, device=DEV)
    has = t % 7 != 3
    lay = ep.Layout(p, send_head=False, recv_src_idx=False)
    pos = torch.where(has, T - 1 - (torch.cumsum(has, 0) - 1), -1)  # the last rows first
    lay.send_pos.copy_(pos.view(1, T, 1))
    ch = torch.arange(H, device=DEV)
    rows = ep.max_recv_rows(p)
    dout = ((t[:, None] * 5 + ch * 3) % 17 - 8).to(torch.bfloat16)
    wt = torch.exp2((t % 5 - 2).float()).view(1, T, 1)
    dy = torch.full((rows, H), 99.0, dtype=torch.bfloat16, device=DEV)
    if mode == ep.MODE_RANK_MAJOR:
        ep.combine_backward(p, lay, dout, None, None, dy=dy)
        wt.fill_(1.0)
    else:
        r = torch.arange(rows, device=DEV)
        y = ((r[:, None] * 7 + ch) % 13 - 6).to(torch.bfloat16)
        dw = torch.full((1, T, 1), float("nan"), device=DEV)
        ep.combine_backward(p, lay, dout, wt, y, dy=dy, dweights=dw)
    torch.cuda.synchronize()
    assert int(lay.err.item()) == 0
    want = torch.full((rows, H), 99.0, dtype=torch.bfloat16, device=DEV)
    want[pos[has]] = (dout.float() * wt.view(T, 1)).to(torch.bfloat16)[has]
    assert torch.equal(dy, want)
    if mode == ep.MODE_NORMAL:
        dot = (dout.float() * y.float()[pos.clamp(min=0)]).sum(1) * has
        assert torch.equal(dw.view(T), dot)
