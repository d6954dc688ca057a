"""Workspace sizes and overlapping outputs of a training step's operators, on the host (nothing is launched)."""
import pytest
import torch

from mixture_experts_grouped_moe_gb300 import build as moe_build

INVALID = -1
P = 1024  # a non-null, aligned stand-in for a device pointer


def refused(fn, good, cases):
    """good: dict of a call; each case changes some arguments."""
    for change, status in cases:
        assert not set(change) - set(good), change
        assert fn(*dict(good, **change).values()) == status, change


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


def test_ffn_output_over_add(moe):
    """out may be add with its pitch, or lie between its rows; every other overlap is refused."""
    lib = moe.load()
    A = 1 << 20  # a stand-in for a device address; only refused calls are made with rows
    good = dict(t=0, act=0, x=P, ld=64, wgu=P, wd=P, add=A, ld_add=64, T=10, H=64, I=32, gu=None, h=None, out=A,
                ld_out=64, ws=P, wsb=1 << 30, st=None)
    refused(lib.moe_ffn, good, [
        (dict(out=A + 16), INVALID), (dict(out=A - 16), INVALID), (dict(out=A + 64 * 2), INVALID),
        (dict(out=A + 9 * 128 + 112), INVALID), (dict(ld_out=72), INVALID), (dict(ld_add=72), INVALID),
        (dict(ld_add=128, ld_out=128, out=A + 112), INVALID), (dict(ld_add=128, ld_out=128, out=A - 112), INVALID),
        (dict(ld_add=128, ld_out=128, out=A + 5 * 256 + 144), INVALID),
        (dict(ld_add=192, ld_out=128, out=A + 128), INVALID), (dict(T=1, out=A + 112), INVALID)])


def test_norm_inside_a_gradient(moe):
    """clip writes the norm while it scales: it cannot lie in a gradient or an output."""
    v = torch.zeros(100)
    clip = moe.GradientClip(1.0, device="cpu")
    for call in (lambda: clip.clip([v], norm=v[3:4]), lambda: clip.clip([v[:50]], [torch.zeros(50)], norm=v[49:50]),
                 lambda: clip.clip([torch.zeros(50)], [v[:50]], norm=v[:1])):
        with pytest.raises(ValueError, match="overlaps"):
            call()
    with pytest.raises(ValueError, match="GPU"):  # (past the checks, as far as a CPU tensor goes)
        clip.clip([v[:50]], norm=v[50:51])
