"""Plain definitions in 64 bits of the norm, the balance loss and the linear
layers, with the e4m3 block cast, for the tests of the CUDA kernels."""
import torch

F8 = torch.float8_e4m3fn


def quantise(y):
    """(values before rounding, scale) of the e4m3 cast of y [rows, 128 n]."""
    b = y.view(y.shape[0], -1, 128)
    scale = b.abs().amax(2).clamp_min(1e-4) / 448
    return (b / scale[:, :, None]).view(y.shape), scale


def e4m3_tolerance(v):
    """Half a step of e4m3 at v, with room for a few fp32 roundings of v: at
    most 2^-4 of the value, and 2^-10 among the subnormals."""
    return torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10) + 1e-4 * v.abs()


def norm(x, res, gamma, eps):
    v = x.double() if res is None else x.double() + res.double()
    rstd = (v.square().mean(1) + eps).rsqrt()
    return v, rstd, v * rstd[:, None] * gamma.double()


def scores(z, score):
    if score == 0:
        return z.softmax(1)
    return torch.nn.functional.logsigmoid(z).softmax(1)


def balance(logits, idx, score, coef, off):
    """loss (differentiable in logits), counts, prob."""
    n, e = logits.shape
    k, s = idx.shape[1], len(off) - 1
    p = scores(logits, score)
    loss = torch.zeros((), dtype=torch.float64, device=logits.device)
    counts = torch.zeros(s, e, dtype=torch.int64, device=logits.device)
    prob = torch.zeros(s, e, dtype=torch.float64, device=logits.device)
    for i in range(s):
        lo, hi = off[i], off[i + 1]
        if lo == hi:
            continue
        ids = idx[lo:hi]
        counts[i] = torch.bincount(ids[(ids >= 0) & (ids < e)].long(), minlength=e)
        mean = p[lo:hi].mean(0)
        prob[i] = mean.detach()
        loss = loss + coef / s * (counts[i].double() * (e / (k * (hi - lo))) * mean).sum()
    return loss, counts, prob


def weight64(w, w_scale, cout):
    """[G, wide, K] weights in 64 bits, e4m3 blocks scaled."""
    if w_scale is None:
        return w.double()
    g, wide, k = w.shape
    s = w_scale.double().view(g, wide // cout, -1, k // 128)
    s = s.repeat_interleave(128, 2)[:, :, :cout].repeat_interleave(128, 3)
    return w.double() * s.reshape(g, wide, k)


def linear(x, x_scale, w, w_scale, bias, act, res, cout):
    """One group: (out, bound of what fp32 sums may be off), in 64 bits. The
    bound holds for sums in steps of 16 products, each step off by at most
    2^-22 of the absolute sum so far, and an epilogue of a few roundings."""
    x = x.double()
    if x_scale is not None:
        x = x * x_scale.double().repeat_interleave(128, 1)
    w = weight64(w[None], None if w_scale is None else w_scale[None], cout)[0]
    z = x @ w.t()
    size = x.abs() @ w.abs().t()
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    err = size * ((x.shape[1] / 16 + 8) * 2.0 ** -22)
    if act == 3:
        g, u, eg, eu = z[:, :cout], z[:, cout:], err[:, :cout], err[:, cout:]
        a = torch.nn.functional.silu(g)
        y, err = a * u, 1.1 * eg * (u.abs() + eu) + a.abs() * eu + (a * u).abs() * 1e-5
    elif act == 1:
        y, err = torch.nn.functional.silu(z), 1.1 * err + z.abs() * 1e-5
    elif act == 2:
        y, err = torch.nn.functional.gelu(z), 1.13 * err + z.abs() * 1e-6
    else:
        y = z
    if res is not None:
        y = y + res.double()
        err = err + y.abs() * 2.0 ** -23
    return y, err


def within(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())
