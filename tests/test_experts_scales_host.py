"""The binding's checks of FP8 scales on the host.  In normal mode scales are
[channels/128][rows] with the row buffer's length as their stride, so a row buffer cut
shorter than its scales would be multiplied with other rows' scales."""
import pytest
import torch

from combine_ep_get_layout_amd import ep

P = dict(R=2, T=8, H=256, E=4, K=2)
u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731


def refused(p, rows, numel, dtype):
    """Whether the binding refuses `numel` scales for [rows][256] codes."""
    try:
        ep._rows(p, u8(rows, 256), "x", 256, torch.zeros(numel, dtype=dtype))
    except ValueError as e:
        if "device tensors" in str(e):  # all that is left to refuse here
            return False
        assert "x scales" in str(e)
        return True
    raise AssertionError("a host tensor was taken")


@pytest.mark.parametrize("dtype", [torch.float32, torch.uint8])
def test_normal_mode_takes_scales_of_the_same_rows_alone(dtype):
    p = ep.Problem(**P)
    assert not refused(p, 32, 2 * 32, dtype)
    for rows, numel in (20, 2 * 32), (32, 2 * 32 + 1), (32, 2 * 32 - 1), (33, 2 * 32), (1, 2 * 32):
        assert refused(p, rows, numel, dtype), (rows, numel)


@pytest.mark.parametrize("mode", [ep.MODE_LOW_LATENCY, ep.MODE_MESSAGES])
def test_blocks_have_a_stride_of_their_own(mode):
    """[E][channels/128][R*T]: the row buffer's length does not matter, too few do."""
    p = ep.Problem(**P, mode=mode)
    for numel in 2 * 64, 2 * 64 + 3:
        assert not refused(p, 64, numel, torch.float32)
        assert not refused(p, 70, numel, torch.float32)
    assert refused(p, 64, 2 * 64 - 1, torch.float32)


def test_no_rows_need_no_scales():
    """A receive buffer without rows keeps one unused scale."""
    r = ep.Recv(ep.Problem(**P, quant=ep.QUANT_FP8_F32), 0, device="cpu")
    assert r.scales.numel() == 1
    assert not refused(ep.Problem(**P), 0, 1, torch.float32)
    assert not refused(ep.Problem(**P), 0, 0, torch.float32)


def test_results_and_short_views():
    """A shortened result with the scales of a whole one; a view of the rows received."""
    p = ep.Problem(**P)
    with pytest.raises(ValueError, match="h scales"):
        ep._rows(p, u8(20, 128), "h", 128, torch.zeros(32))
    recv = ep.Recv(ep.Problem(**P, quant=ep.QUANT_FP8_F32), 32, device="cpu")
    with pytest.raises(ValueError, match="x scales"):
        ep._rows(p, recv.x[:20], "x", 256, recv.scales)
