"""Arguments that the norm, balance-loss and linear calls refuse, on the host
and before any launch (these run without a GPU)."""
import ctypes

import pytest
import torch

from combine_top_group_b200 import ep

A = 1 << 20  # an aligned address that nothing reads


def status(fn, *a):
    return getattr(ep._lib, fn)(*a)


NORM = dict(N=4, H=256, x=A, res=None, gamma=A, gt=0, eps=1e-6, h=None, y=A, q=None, qs=None, rstd=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(N=-1), 1), (dict(N=1 << 31), 5), (dict(H=0), 5), (dict(H=100), 5), (dict(H=65664), 5), (dict(gt=2), 1),
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(x=None), 1), (dict(gamma=None), 1),
    (dict(y=None), 1), (dict(q=A), 1), (dict(qs=A), 1), (dict(h=A), 1), (dict(x=A + 16), 1), (dict(res=A + 2), 1),
    (dict(gamma=A + 4), 1), (dict(y=A + 16), 1), (dict(q=A + 8, qs=A), 1), (dict(q=A, qs=A + 2), 1),
    (dict(rstd=A + 1), 1), (dict(h=A + 64 + 8), 1)])
def test_norm(change, want):
    assert status("ep_rmsnorm", *{**NORM, **change}.values()) == want
    assert ep.ep_last_error_message()


BACK = dict(N=4, H=256, h=A, rstd=A, gamma=A, gt=0, dy=A, dh=None, dx=A, dg=A, ws=A, bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(N=-1), 1), (dict(H=130), 5), (dict(gt=-1), 1), (dict(h=None), 1), (dict(rstd=None), 1), (dict(gamma=None), 1),
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(dg=None), 1), (dict(ws=None), 1), (dict(ws=A + 128), 1),
    (dict(bytes=4 * 256 * 4 - 1), 3), (dict(h=A + 8), 1), (dict(dh=A + 8), 1), (dict(dg=A + 2), 1)])
def test_norm_backward(change, want):
    assert status("ep_rmsnorm_backward", *{**BACK, **change}.values()) == want
    assert ep.ep_last_error_message()


LOSS = dict(N=64, E=16, K=2, score=0, logits=A, idx=A, S=1, off=None, coef=1.0, loss=A, counts=A, prob=None, ws=A,
            bytes=1 << 30, err=A, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(N=-1), 1), (dict(N=1 << 31), 5), (dict(E=0), 5), (dict(E=1025), 5), (dict(K=0), 1), (dict(K=17), 1),
    (dict(E=64, K=33), 1), (dict(score=2), 1), (dict(score=-1), 1), (dict(logits=None), 1), (dict(idx=None), 1),
    (dict(S=0), 1), (dict(S=2), 1), (dict(S=(1 << 24) + 1, off=A), 5), (dict(off=A + 2), 1), (dict(loss=None), 1),
    (dict(counts=None), 1), (dict(err=None), 1), (dict(ws=None), 1), (dict(ws=A + 64), 1), (dict(bytes=256), 3),
    (dict(logits=A + 2), 1), (dict(prob=A + 1), 1)])
def test_balance(change, want):
    assert status("ep_balance_loss", *{**LOSS, **change}.values()) == want
    assert ep.ep_last_error_message()


GRAD = dict(N=64, E=16, K=2, score=0, logits=A, S=1, off=None, counts=A, coef=1.0, g=None, acc=0, dz=A, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(N=-1), 1), (dict(E=1025), 5), (dict(K=17), 1), (dict(score=5), 1), (dict(logits=None), 1), (dict(S=3), 1),
    (dict(counts=None), 1), (dict(dz=None), 1), (dict(g=A + 1), 1), (dict(dz=A + 2), 1)])
def test_balance_backward(change, want):
    assert status("ep_balance_loss_backward", *{**GRAD, **change}.values()) == want
    assert ep.ep_last_error_message()


def test_workspace_sizes():
    for fn in (lambda: ep.ep_rmsnorm_backward_workspace_bytes(-1, 256),
               lambda: ep.ep_rmsnorm_backward_workspace_bytes(4, 257),
               lambda: ep.ep_balance_loss_workspace_bytes(-1, 8), lambda: ep.ep_balance_loss_workspace_bytes(4, 0),
               lambda: ep.ep_balance_loss_workspace_bytes(4, 8, 0)):
        with pytest.raises(ep.EpError):
            fn()
    assert ep.ep_rmsnorm_backward_workspace_bytes(0, 256) > 0 and ep.ep_balance_loss_workspace_bytes(0, 8) > 0
    # bounded in the rows: partial sums, not one per row
    assert ep.ep_rmsnorm_backward_workspace_bytes(1 << 30, 7168) < 1 << 26


def test_linear_without_buffer():
    a = ep.EpLinear()
    assert ep._lib.ep_linear(None, 1, ctypes.byref(a), None) == ep.EP_ERR_INVALID
    assert ep._lib.ep_expert_linear(None, 1, ctypes.byref(a), None) == ep.EP_ERR_INVALID


def test_host_tensors_are_refused():
    x, g = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    with pytest.raises(ep.EpError):
        ep.ep_rmsnorm(x, g, 1e-6, y=torch.empty_like(x))
    with pytest.raises(ep.EpError):
        ep.ep_rmsnorm_backward(x, torch.zeros(4), g, x, x.clone(), torch.zeros(256), torch.zeros(1 << 16, dtype=torch.uint8))
    z = torch.zeros(4, 16)
    with pytest.raises(ep.EpError):
        ep.ep_balance_loss(z, torch.zeros(4, 2, dtype=torch.int32), 0, 1.0, torch.zeros(1),
                           torch.zeros(1, 16, dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.uint8),
                           torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ep.EpError):
        ep.ep_balance_loss_backward(z, torch.zeros(1, 16, dtype=torch.int32), 2, 0, 1.0, z.clone())


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: nothing may be launched on them")
def test_norm_without_a_device():
    """Where the device cannot be asked what it holds at once, the call fails
    there. (It does not fall back to a kernel that adds up in another order.)"""
    big = dict(N=100000, H=256)
    assert status("ep_rmsnorm", *{**NORM, **big}.values()) == ep.EP_ERR_CUDA
    assert "resident CTAs" in ep.ep_last_error_message()
    assert status("ep_rmsnorm_backward", *{**BACK, **big}.values()) == ep.EP_ERR_CUDA
    assert "resident CTAs" in ep.ep_last_error_message()
