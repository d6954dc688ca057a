"""Workspace sizes and overlapping outputs of a training step's operators, on the host (nothing is launched)."""
import pytest

from mixture_experts_grouped_moe_gb300 import build as moe_build

INVALID = -1
P = 1024  # a non-null, aligned stand-in for a device pointer


@pytest.fixture(scope="module")
def moe():
    moe_build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


def test_workspace_of_the_loss_covers_smaller_batches(moe):
    """A workspace for T rows serves every smaller T (and V, as far as the forward goes)."""
    size = moe.moe_vocab_loss_workspace_size
    for H in (64, 4096):
        for V in (1, 300, 2000, 9729, 32000, 128001):
            for piece in (0, 64, 8192):
                last = 0
                for T in list(range(0, 300)) + [1000, 9728, 9729, 20000]:
                    now = size(T, H, V, piece)
                    assert now >= last, (H, V, piece, T)
                    last = now
    for T in (1, 16, 32, 33, 256, 1000):
        sizes = [size(T, 64, V) for V in range(1, 40000, 101)]
        assert sizes == sorted(sizes), T

