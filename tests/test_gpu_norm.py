"""ep_rmsnorm and its gradient against the definition in 64 bits.

Tolerances: half a step of the output's type, plus 2^-14 of the value for the
fp32 sum of squares (at most about 100 sequential additions per thread and
tree level, 2^-24 each, halved by the root) and the products after it."""
import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = 2.0 ** -8 * 1.001  # bf16: half a step, and the fp32 roundings before it
SUMS = 2.0 ** -14


@pytest.fixture(scope="module")
def ep():
    from combine_top_group_b200 import ep as m
    return m


def rand(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def guard(dtype, *shape):
    """An output followed by a canary row: (whole, view without the canary)."""
    whole = torch.full((shape[0] + 1, *shape[1:]), 7.0, device=DEV).to(dtype)
    return whole, whole[:-1]


def untouched(whole):
    assert (whole[-1].float() == 7.0).all()


SHAPES = [(1, 128), (1, 7168), (3, 256), (33, 384), (7, 512), (5, 640), (130, 1024), (2, 4224), (9, 8192), (3, 8320),
          (2, 16384), (2, 32768), (1, 32896), (2, 65536), (1025, 128)]


@pytest.mark.parametrize("n,h", SHAPES)
@pytest.mark.parametrize("gamma_type", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_forward(ep, n, h, gamma_type, residual):
    x, res = rand(1, n, h, scale=1.5), rand(2, n, h) if residual else None
    gamma = 1 + rand(3, h, dtype=gamma_type, scale=0.2)
    hw, ho = guard(BF, n, h)
    yw, y = guard(BF, n, h)
    qw, q = guard(F8, n, h)
    sw, scale = guard(F32, n, h // 128)
    rw, rstd = guard(F32, n)
    ep.ep_rmsnorm(x, gamma, 1e-6, residual=res, h=ho, y=y, q=q, q_scale=scale, rstd=rstd)
    v, r64, n64 = ref.norm(x, res, gamma, 1e-6)
    ref.within(ho, v, v.abs() * HALF, "h")
    ref.within(rstd, r64, r64 * SUMS, "rstd")
    ref.within(y, n64, n64.abs() * (HALF + SUMS), "y")
    q64, s64 = ref.quantise(n64)
    ref.within(scale, s64, s64 * SUMS, "q_scale")
    ref.within(q.float(), q64, ref.e4m3_tolerance(q64), "q")
    for w in (hw, yw, qw, sw, rw):
        untouched(w)


@pytest.mark.parametrize("n,h", [(37889, 128), (20000, 256), (9500, 384), (9473, 512), (4800, 640), (4737, 1024), (1300, 2176),
                                 (700, 7168), (3000, 7168), (601, 8192), (700, 8320), (600, 16384), (1201, 12416)])
@pytest.mark.parametrize("residual", [False, True])
def test_forward_on_many_rows(ep, n, h, residual):
    """Rows enough for persistent CTAs that stream them."""
    test_forward(ep, n, h, F32, residual)
    if n * h < 1 << 23:
        test_forward(ep, n, h, BF, residual)


@pytest.mark.parametrize("outputs", [("h",), ("y",), ("q", "q_scale"), ("rstd",), ("h", "q", "q_scale")])
def test_any_outputs(ep, outputs):
    """Each set of outputs gives the bits that all of them together give."""
    n, h = 19, 896
    x, res, gamma = rand(1, n, h), rand(2, n, h), rand(3, h)
    full = dict(h=torch.empty(n, h, dtype=BF, device=DEV), y=torch.empty(n, h, dtype=BF, device=DEV),
                q=torch.empty(n, h, dtype=F8, device=DEV), q_scale=torch.empty(n, h // 128, device=DEV),
                rstd=torch.empty(n, device=DEV))
    ep.ep_rmsnorm(x, gamma, 1e-5, residual=res, **full)
    some = {k: torch.empty_like(full[k]) for k in outputs}
    ep.ep_rmsnorm(x, gamma, 1e-5, residual=res, **some)
    for k in outputs:
        assert torch.equal(some[k].view(torch.uint8), full[k].view(torch.uint8)), k


def test_quantised_as_dispatch_does(ep):
    """q and q_scale are what dispatch writes for the same values: the norm of
    rows whose normalised values are bf16 numbers."""
    n, h = 16, 512
    y = torch.randint(0, 2, (n, h), generator=torch.Generator().manual_seed(0)).float().to(DEV) * 2 - 1  # +-1: rms is 1
    q, s = torch.empty(n, h, dtype=F8, device=DEV), torch.empty(n, h // 128, device=DEV)
    gamma = rand(5, h)
    ep.ep_rmsnorm(y.to(BF), gamma, 1e-30, q=q, q_scale=s)
    cfg = ep.ep_default_config(1, n, h, 4, 1)
    cfg.flags = ep.EP_FLAG_FP8
    buf = ep.ep_buffer_create(cfg, device=DEV)
    ep.ep_get_layout(buf, n, topk_idx=torch.zeros(n, 1, dtype=torch.int32, device=DEV),
                     topk_w=torch.ones(n, 1, device=DEV))
    ep.ep_dispatch(buf, n, (y * gamma.float()).to(BF).contiguous())
    recv = ep.ep_buffer_recv(buf)
    assert torch.equal(recv["recv_x"][:n], q.view(torch.uint8))
    assert torch.equal(recv["recv_scale"][:n], s)


def test_rows_without_scale(ep):
    """Zero rows, rows of the type's largest values and rows with infinities
    or NaN stay apart from their neighbours."""
    n, h = 6, 256
    x, gamma = rand(1, n, h), torch.ones(h, device=DEV)
    x[0] = 0
    x[1] = 3.38e38   # squares overflow fp32: rstd 0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4] = 1e-30     # squares underflow: eps alone
    y, q, s = torch.empty(n, h, dtype=BF, device=DEV), torch.empty(n, h, dtype=F8, device=DEV), \
        torch.empty(n, h // 128, device=DEV)
    r = torch.empty(n, device=DEV)
    ep.ep_rmsnorm(x, gamma, 1e-6, y=y, q=q, q_scale=s, rstd=r)
    assert (y[0] == 0).all() and (q[0].float() == 0).all()
    ref.within(s[0], torch.full((2,), 1e-4 / 448, dtype=torch.float64, device=DEV), 1e-12, "floor of the scale")
    assert (y[1] == 0).all() and r[1] == 0
    assert y[2, 5].isnan() and (y[2, 6:] == 0).all()
    assert y[3].isnan().all()
    ref.within(y[4], x[4].double() * 1e3, 1e-27 * 2.0 ** -7, "underflow")
    _, _, n64 = ref.norm(x[5:], None, gamma, 1e-6)
    ref.within(y[5:], n64, n64.abs() * (HALF + SUMS), "neighbour")


@pytest.mark.parametrize("place", ["x", "residual"])
def test_in_place(ep, place):
    n, h = 70, 1152
    x, res, gamma = rand(1, n, h), rand(2, n, h), rand(3, h)
    ho, y = torch.empty_like(x), torch.empty_like(x)
    ep.ep_rmsnorm(x, gamma, 1e-6, residual=res, h=ho, y=y)
    a = dict(x=x.clone(), residual=res.clone())
    y2 = a["residual" if place == "x" else "x"]
    ep.ep_rmsnorm(a["x"], gamma, 1e-6, residual=a["residual"], h=a[place], y=y2)
    assert torch.equal(a[place], ho) and torch.equal(y2, y)


BACK = [(20000, 128), (5000, 1536), (1500, 7168), (700, 12416), (1, 128), (2, 7168), (517, 1024), (40, 384), (3, 8320), (2, 65536), (3000, 256), (1, 4096)]


@pytest.mark.parametrize("n,h", BACK)
@pytest.mark.parametrize("gamma_type", [BF, F32])
@pytest.mark.parametrize("dh", [False, True])
def test_backward(ep, n, h, gamma_type, dh):
    x, dy = rand(1, n, h, scale=1.5), rand(2, n, h)
    gamma = 1 + rand(3, h, dtype=gamma_type, scale=0.2)
    inc = rand(4, n, h) if dh else None
    rstd = torch.empty(n, device=DEV)
    ep.ep_rmsnorm(x, gamma, 1e-6, rstd=rstd)
    dxw, dx = guard(BF, n, h)
    dgw = torch.full((h + 32,), 7.0, device=DEV)
    size = ep.ep_rmsnorm_backward_workspace_bytes(n, h)
    ws = torch.full((size + 64,), 0x5a, dtype=torch.uint8, device=DEV)
    ep.ep_rmsnorm_backward(x, rstd, gamma, dy, dx, dgw[:h], ws[:size], dh=inc)
    r, t = rstd.double()[:, None], dy.double() * gamma.double()
    nn = x.double() * r
    m = (t * nn).mean(1, keepdim=True)
    want = r * (t - nn * m) + (inc.double() if dh else 0)
    size_of = r * (t.abs() + nn.abs() * (t * nn).abs().mean(1, keepdim=True)) + (inc.double().abs() if dh else 0)
    ref.within(dx, want, want.abs() * HALF + size_of * SUMS, "dx")
    # a slot's rows in order, then at most 1184 slots in 8 strides
    ref.within(dgw[:h], (dy.double() * nn).sum(0), (dy.double() * nn).abs().sum(0) * (n + 200) * 2.0 ** -24, "dgamma")
    untouched(dxw)
    assert (dgw[h:] == 7).all() and (ws[size:] == 0x5a).all()


def test_backward_against_differences(ep):
    """The kernel's gradient against differences of the definition, through
    the norm with a residual."""
    n, h = 3, 256
    x, res, gamma, dy = rand(1, n, h), rand(2, n, h), 1 + rand(3, h, dtype=F32, scale=0.2), rand(4, n, h)
    ho, rstd = torch.empty_like(x), torch.empty(n, device=DEV)
    ep.ep_rmsnorm(x, gamma, 1e-6, residual=res, h=ho, rstd=rstd)
    dx, dg = torch.empty_like(x), torch.empty(h, device=DEV)
    ws = torch.empty(ep.ep_rmsnorm_backward_workspace_bytes(n, h), dtype=torch.uint8, device=DEV)
    ep.ep_rmsnorm_backward(ho, rstd, gamma, dy, dx, dg, ws)
    v = ho.double()

    def loss(v, g):
        return (v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt() * g * dy.double()).sum()
    for seed in range(4):
        d = rand(10 + seed, n, h, dtype=torch.float64)
        e = 1e-5
        slope = (loss(v + e * d, gamma.double()) - loss(v - e * d, gamma.double())) / (2 * e)
        # each of the n*h terms is off by a bf16 half step of dx
        tol = (dx.double() * d).abs().sum() * 2.0 ** -7
        assert abs((dx.double() * d).sum() - slope) <= tol
        dgd = rand(20 + seed, h, dtype=torch.float64)
        slope = (loss(v, gamma.double() + e * dgd) - loss(v, gamma.double() - e * dgd)) / (2 * e)
        # rstd is that of the sum before its rounding to h = v (1 + d), |d| <= 2^-8. So mean(h^2) is off by at
        # most a factor (1 + 2^-8)^2, rstd and with it every term of the kernel's dgamma by 1 + 2^-8, and the
        # terms' fp32 products by far less. Terms of opposite sign in a column keep their own size.
        terms = (dy.double() * v * rstd.double()[:, None] * dgd).abs().sum()
        assert abs((dg.double() * dgd).sum() - slope) <= terms * (2.0 ** -8 * 1.001)


@pytest.mark.parametrize("place", ["dy", "dh"])
def test_backward_in_place(ep, place):
    n, h = 300, 640
    x, gamma = rand(1, n, h), rand(3, h)
    a = dict(dy=rand(2, n, h), dh=rand(4, n, h))
    rstd = torch.empty(n, device=DEV)
    ep.ep_rmsnorm(x, gamma, 1e-6, rstd=rstd)
    ws = torch.empty(ep.ep_rmsnorm_backward_workspace_bytes(n, h), dtype=torch.uint8, device=DEV)
    dx, dg, dg2 = torch.empty_like(x), torch.empty(h, device=DEV), torch.empty(h, device=DEV)
    ep.ep_rmsnorm_backward(x, rstd, gamma, a["dy"], dx, dg, ws, dh=a["dh"])
    ep.ep_rmsnorm_backward(x, rstd, gamma, a["dy"], a[place], dg2, ws, dh=a["dh"])
    assert torch.equal(a[place], dx) and torch.equal(dg, dg2)


def test_no_rows(ep):
    h = 256
    x, gamma = torch.empty(0, h, dtype=BF, device=DEV), rand(1, h)
    ep.ep_rmsnorm(x, gamma, 1e-6, y=torch.empty_like(x))
    dg = torch.full((h,), 3.0, device=DEV)
    ws = torch.empty(ep.ep_rmsnorm_backward_workspace_bytes(0, h), dtype=torch.uint8, device=DEV)
    ep.ep_rmsnorm_backward(x, torch.empty(0, device=DEV), gamma, x, torch.empty_like(x), dg, ws)
    assert (dg == 0).all()


def test_offsets_past_32_bits(ep):
    """The last rows of arrays that hold more than 2^31 channels."""
    h = 65536
    n = 2 ** 31 // h + 3
    x = torch.zeros(n, h, dtype=BF, device=DEV)
    x[-2:] = rand(1, 2, h)
    gamma = rand(2, h)
    y = torch.empty_like(x)
    ep.ep_rmsnorm(x, gamma, 1e-6, y=y)
    _, _, n64 = ref.norm(x[-2:], None, gamma, 1e-6)
    ref.within(y[-2:], n64, n64.abs() * (HALF + SUMS), "y")
    assert (y[:4] == 0).all()


def test_graph_and_streams(ep):
    """Captured and replayed on new inputs, and run at once on two streams with
    a workspace each, the calls give the bits of plain ones."""
    n, h = 257, 2048
    gamma = rand(3, h)
    ws = [torch.empty(ep.ep_rmsnorm_backward_workspace_bytes(n, h), dtype=torch.uint8, device=DEV) for _ in range(2)]

    def step(s, st=None):
        ep.ep_rmsnorm(s["x"], gamma, 1e-6, residual=s["r"], h=s["h"], y=s["y"], rstd=s["rstd"], stream=st)
        ep.ep_rmsnorm_backward(s["h"], s["rstd"], gamma, s["dy"], s["dx"], s["dg"], ws[s["w"]], dh=s["r"], stream=st)

    def state(seed, w):
        x = rand(seed, n, h)
        return dict(x=x, r=rand(seed + 1, n, h), dy=rand(seed + 2, n, h), h=torch.empty_like(x), y=torch.empty_like(x),
                    dx=torch.empty_like(x), rstd=torch.empty(n, device=DEV), dg=torch.empty(h, device=DEV), w=w)
    a, b = state(1, 0), state(11, 1)
    step(a), step(b)
    want = [{k: s[k].clone() for k in ("h", "y", "dx", "dg")} for s in (a, b)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    for k in ("x", "r", "dy"):
        a[k].copy_(b[k])
    g.replay()
    torch.cuda.synchronize()
    for k, t in want[1].items():
        assert torch.equal(a[k], t), k
    a = state(1, 0)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        step(a, s1), step(b, s2)
    torch.cuda.synchronize()
    for s, w in ((a, want[0]), (b, want[1])):
        for k, t in w.items():
            assert torch.equal(s[k], t), k


@pytest.mark.parametrize("n,h", [(700, 16512), (1300, 32896), (601, 65536)])
def test_backward_of_many_long_rows(ep, n, h):
    """Rows too long for the streams, several to a CTA."""
    test_backward(ep, n, h, F32, True)
    test_backward(ep, n, h, BF, False)
