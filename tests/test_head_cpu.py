"""The head's workspace holds what its calls use, and no more."""
import pytest

import token_routing_expert_router_gb300 as moe


@pytest.fixture(autouse=True)
def _built(lib):
    pass


def size(**kw):
    return moe.moe_head_workspace_size(moe.MoEHeadConfig.make(**kw))


def padded(n, to):
    return -(-n // to) * to


def test_no_room_for_splits_that_cannot_be():
    """A vocabulary of 16 K stages is never split: x's rows that count, dz and the tiles' sums alone."""
    T, H, V = 4096, 4096, 1000
    x, dz, part = T * H * 2, T * 1024 * 2, 8 * 2 * T * 8
    assert x + dz + part <= size(T=T, H=H, V=V) < x + dz + part + T * 16 + (1 << 16)


def test_one_plane_of_bf16_rows_of_odd_width():
    """They are laid out once each; only dz has three planes."""
    T, H, V = 4096, 1001, 2000
    Hp, piece = padded(H, 8), padded(V, 256)
    x, w, dz, part = T * Hp * 2, piece * Hp * 2, 3 * T * piece * 2, 16 * 2 * T * 8
    slices = 4 * 76 * 256 * 128 * 4
    assert x + w + dz + part <= size(T=T, H=H, V=V) < x + w + dz + part + slices + T * 16 + (1 << 16)


def test_three_planes_of_fp32_rows():
    T, H, V = 4096, 1000, 2000
    piece = padded(V, 256)
    x, w, dz, part = 3 * T * H * 2, 3 * piece * H * 2, 3 * T * piece * 2, 16 * 2 * T * 8
    slices = 4 * 76 * 256 * 128 * 4
    assert x + w + dz + part <= size(T=T, H=H, V=V, act_dtype=moe.F32) < x + w + dz + part + slices + T * 16 + (1 << 16)
