"""How tv_prefill cuts prompts (the workspace that it asks for holds a state and a decay for each
segment), at sizes where both sides were measured on 152 SMs."""
import pytest

import tree_speculative_verify_tv_gb300 as tv


def pieces(B, H, rows, dk, dv):
    size = tv.tv_prefill_workspace_bytes(B, B * rows, rows, H, dk, dv, tv.TV_DECAY_SCALAR, tv.TV_BF16)
    return max(1, size // (B * H * (dk * dv * 4 + 8)))


@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 128), (64, 64)])
@pytest.mark.parametrize("B,H,rows,want", [
    (1, 32, 32768, 9),   # 395 us (4 pieces 466, 28 463, at an earlier step)
    (2, 32, 16384, 7),   # 412 us at 128 x 128, in 2 pieces 456; 64 x 64: 294 and 344
    (1, 64, 16384, 7),   # 416 and 458; 300 and 351
    (1, 64, 4096, 1),    # 98 us at 64 x 64 uncut, in 2 pieces 104; 128 x 128: 144 and 138
    (8, 32, 4096, 1)])
def test_segments_of_long_prompts(B, H, rows, want, dk, dv):
    assert pieces(B, H, rows, dk, dv) == want
