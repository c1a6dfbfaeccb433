"""ep_balance_loss and its gradient against the definition in 64 bits (the
gradient by torch's autograd of that definition, and by differences).

Tolerances: __expf is off by 2 + 1.173 |x| ulp (2^-23), so 15 ulp where |x| is
about 11, the largest difference of two normal logits here; sums over E and
over tokens, and the products after them, add under 40 roundings of 2^-24. So
2^-18 relative covers a score, and 2^-17 a sum of products of two scores."""
import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 2.0 ** -17


@pytest.fixture(scope="module")
def ep():
    from combine_top_group_b200 import ep as m
    return m


def case(seed, n, e, k, mask=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = torch.randn(n, e, generator=g, device=DEV)
    idx = z.topk(k, dim=1).indices.int()
    drop = torch.rand(n, k, generator=g, device=DEV) < mask
    return z, torch.where(drop, -1, idx).contiguous()


def run(ep, z, idx, score, coef, off, grad=None, accumulate=None, prob=True, error=0):
    n, e = z.shape
    s = len(off) - 1 if off is not None else 1
    o = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    loss, counts = torch.full((2,), 7.0, device=DEV), torch.full((s + 1, e), 7, dtype=torch.int32, device=DEV)
    pr = torch.full((s + 1, e), 7.0, device=DEV)
    size = ep.ep_balance_loss_workspace_bytes(n, e, s)
    ws = torch.full((size + 64,), 0x5a, dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ep.ep_balance_loss(z, idx, score, coef, loss[:1], counts[:s], ws[:size], err, seq_off=o, prob=pr[:s] if prob else None)
    dz = torch.full_like(z, 7.0) if accumulate is None else accumulate.clone()
    ep.ep_balance_loss_backward(z, counts[:s], idx.shape[1], score, coef, dz, seq_off=o, grad_loss=grad,
                                accumulate=accumulate is not None)
    assert err.item() == error
    assert loss[1] == 7 and (counts[s] == 7).all() and (pr[s] == 7).all() and (ws[size:] == 0x5a).all()
    return loss[0], counts[:s], pr[:s], dz


SHAPES = [(1, 1, 1), (1, 8, 2), (5, 3, 3), (9, 32, 4), (64, 33, 8), (100, 64, 6), (37, 100, 5), (129, 128, 8), (50, 130, 7),
          (300, 256, 8), (31, 257, 3), (40, 384, 8), (21, 513, 2), (70, 1024, 32), (19, 1023, 9), (2500, 16, 2)]


@pytest.mark.parametrize("n,e,k", SHAPES)
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("packed", [False, True])
def test_loss_and_gradient(ep, n, e, k, score, packed):
    z, idx = case(n + e, n, e, k, 0.2)
    off = sorted({0, n // 3, n // 3 + 1, 2 * n // 3}) + [n, n] if packed else [0, n]  # an empty one at the end
    grad = torch.tensor([1.75], device=DEV)
    loss, counts, prob, dz = run(ep, z, idx, score, 0.125, off if packed else None, grad)
    z64 = z.double().requires_grad_()
    l64, c64, p64 = ref.balance(z64, idx, score, 0.125, off)
    (l64 * 1.75).backward()
    assert torch.equal(counts.long(), c64)
    ref.within(prob, p64, p64 * REL, "prob")
    assert abs(loss.double() - l64) <= l64.abs() * REL + 1e-30
    # each entry is g p (f - sum f p): off by REL of g p (f + sum f p)
    p = ref.scores(z.double(), score)
    size = torch.zeros_like(p)
    for i in range(len(off) - 1):
        lo, hi = off[i], off[i + 1]
        if lo < hi:
            f = c64[i].double() * e / (k * (hi - lo))
            size[lo:hi] = p[lo:hi] * (f + (p[lo:hi] * f).sum(1, keepdim=True)) * (1.75 * 0.125 / (len(off) - 1) / (hi - lo))
    ref.within(dz, z64.grad, size * REL + 1e-30, "dlogits")


def test_gradient_against_differences(ep):
    n, e, k = 12, 24, 3
    z, idx = case(5, n, e, k, 0.3)
    off = [0, 5, 5, 12]
    for score in (0, 1):
        _, _, _, dz = run(ep, z, idx, score, 1.0, off)
        for seed in range(3):
            d = torch.randn(n, e, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).double()
            h = 1e-5
            up, down = (ref.balance(z.double() + s * h * d, idx, score, 1.0, off)[0] for s in (1, -1))
            assert abs((dz.double() * d).sum() - (up - down) / (2 * h)) <= (dz.double() * d).abs().sum() * 1e-4


@pytest.mark.parametrize("score", [0, 1])
def test_many_sequences(ep, score):
    """More sequences than CTAs, most of one token, runs of empty ones, and
    sequences that end inside a CTA's chunk."""
    n, e, k = 6000, 64, 6
    z, idx = case(1, n, e, k, 0.05)
    g = torch.Generator().manual_seed(0)
    cuts = torch.randint(0, n + 1, (5000,), generator=g).sort().values.tolist()
    off = [0] + cuts + [n]
    loss, counts, prob, dz = run(ep, z, idx, score, 1.0, off)
    z64 = z.double().requires_grad_()
    l64, c64, p64 = ref.balance(z64, idx, score, 1.0, off)
    l64.backward()
    assert torch.equal(counts.long(), c64)
    ref.within(prob, p64, p64 * REL, "prob")
    assert abs(loss.double() - l64) <= l64 * REL
    ref.within(dz, z64.grad, z64.grad.abs() * 1e-3 + z64.grad.abs().max() * REL, "dlogits")


def test_rows_outside_the_sequences(ep):
    """Padding before and after the sequences is read by nothing and written
    by nothing, even where it holds NaN and ids out of range."""
    n, e, k = 90, 48, 4
    z, idx = case(2, n, e, k)
    z[:7], z[80:] = float("nan"), float("inf")
    idx[:7], idx[80:] = 10 ** 6, -5
    off = [7, 30, 80]
    loss, counts, prob, dz = run(ep, z, idx, 0, 1.0, off)
    l64, c64, p64 = ref.balance(z[7:80].double(), idx[7:80], 0, 1.0, [0, 23, 73])
    assert torch.equal(counts.long(), c64) and abs(loss.double() - l64) <= l64 * REL
    assert (dz[:7] == 7).all() and (dz[80:] == 7).all() and dz[7:80].isfinite().all()


def test_masked_tokens(ep):
    """Tokens whose slots are all masked count towards the mean scores only; with
    no slot at all the loss and the gradient are 0."""
    n, e, k = 20, 16, 2
    z, idx = case(3, n, e, k)
    idx[:] = -1
    loss, counts, prob, dz = run(ep, z, idx, 1, 1.0, None)
    assert loss == 0 and (counts == 0).all() and (dz == 0).all()
    p64 = ref.scores(z.double(), 1).mean(0)
    ref.within(prob[0], p64, p64 * REL, "prob")


def test_bad_ids(ep):
    n, e, k = 40, 16, 2
    z, idx = case(3, n, e, k)
    bad = idx.clone()
    bad[3, 0], bad[9, 1] = 16, -2
    masked = torch.where((bad < 0) | (bad >= e), -1, bad).contiguous()
    a, b = run(ep, z, bad, 0, 1.0, None, error=ep.EP_DEVERR_EXPERT_ID), run(ep, z, masked, 0, 1.0, None)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("off", [[0, 30, 20, 40], [-4, 10, 20, 40], [0, 10, 20, 2 ** 31 - 1], [40, 30, 20, 0],
                                 [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, -2 ** 31]])
def test_bad_offsets(ep, off):
    """Offsets out of order or range are reported and reach no other memory
    (the canaries in run)."""
    z, idx = case(3, 40, 16, 2)
    run(ep, z, idx, 0, 1.0, off, error=ep.EP_DEVERR_ROW_BOUNDS)


@pytest.mark.parametrize("score", [0, 1])
def test_extreme_logits(ep, score):
    """Logits far apart, all far below or above zero: the scores stay a
    distribution."""
    n, e, k = 8, 40, 3
    z, idx = case(4, n, e, k)
    z[1] -= 300
    z[2] += 300
    z[3, 5] = 1e30
    z[4] = -1e30
    z[5] *= 30
    z[6] -= 45
    loss, counts, prob, dz = run(ep, z, idx, score, 1.0, list(range(n + 1)))
    p64 = ref.scores(z.double(), score)
    # |z - max| reaches 200 in row 5: 2 + 1.173 * 200 ulp on terms of at most exp(-|z - max|)
    ref.within(prob, p64, p64 * 2.0 ** -14 + 1e-30, "prob")
    assert dz.isfinite().all()


def test_accumulate_and_scale(ep):
    n, e, k = 77, 72, 4
    z, idx = case(6, n, e, k)
    _, _, _, a = run(ep, z, idx, 1, 0.5, [0, 40, 77])
    base = torch.randn(n, e, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    _, _, _, b = run(ep, z, idx, 1, 0.5, [0, 40, 77], accumulate=base)
    ref.within(b, base.double() + a.double(), (base + a).abs().double() * 2.0 ** -23, "accumulated")
    _, _, _, c = run(ep, z, idx, 1, 0.5, [0, 40, 77], grad=torch.tensor([2.0], device=DEV))
    assert torch.equal(c, 2 * a)


def test_unaligned_rows(ep):
    """Logits that start 4 bytes into an allocation take the scalar loads."""
    n, e, k = 33, 64, 4
    z, idx = case(7, n, e, k)
    whole = torch.empty(n * e + 1, device=DEV)
    z2 = whole[1:].view(n, e)
    z2.copy_(z)
    a, b = run(ep, z, idx, 0, 1.0, None), run(ep, z2, idx, 0, 1.0, None)
    assert torch.equal(a[1], b[1])
    ref.within(a[2], b[2].double(), b[2].double() * REL, "prob")


def test_no_tokens(ep):
    z, idx = torch.empty(0, 16, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    loss, counts, prob, _ = run(ep, z, idx, 0, 1.0, [0, 0, 0])
    assert loss == 0 and (counts == 0).all() and (prob == 0).all()


def test_offsets_past_32_bits(ep):
    n, e, k = 2 ** 21 + 100, 1024, 1
    z = torch.zeros(n, e, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(0)
    z[-64:] = torch.randn(64, e, generator=g, device=DEV)
    idx = torch.zeros(n, k, dtype=torch.int32, device=DEV)
    off = [0, n - 64, n]
    loss, counts, prob, dz = run(ep, z, idx, 0, 1.0, off)
    p64 = z[-64:].double().softmax(1).mean(0)
    ref.within(prob[1], p64, p64 * REL, "prob")
    assert counts[0, 0] == n - 64 and counts[1, 0] == 64
    f, p = 1024.0, z[-64:].double().softmax(1)
    want = p * ((torch.arange(e, device=DEV) == 0) * f - p[:, :1] * f) / 2 / 64
    ref.within(dz[-64:], want, p * f * (1 + p[:, :1]) / 128 * REL, "dlogits")


def test_graph_and_streams(ep):
    n, e, k = 3000, 256, 8
    off = torch.tensor([0, 100, 2900, 3000], dtype=torch.int32, device=DEV)

    def state(seed):
        z, idx = case(seed, n, e, k)
        return dict(z=z, idx=idx, loss=torch.empty(1, device=DEV), counts=torch.empty(3, e, dtype=torch.int32, device=DEV),
                    prob=torch.empty(3, e, device=DEV), dz=torch.empty(n, e, device=DEV),
                    ws=torch.empty(ep.ep_balance_loss_workspace_bytes(n, e, 3), dtype=torch.uint8, device=DEV),
                    err=torch.zeros(1, dtype=torch.int32, device=DEV))

    def step(s, st=None):
        ep.ep_balance_loss(s["z"], s["idx"], 0, 0.01, s["loss"], s["counts"], s["ws"], s["err"], seq_off=off, prob=s["prob"], stream=st)
        ep.ep_balance_loss_backward(s["z"], s["counts"], k, 0, 0.01, s["dz"], seq_off=off, stream=st)
    a, b = state(1), state(2)
    step(a), step(b)
    names = ("loss", "counts", "prob", "dz")
    want = [{x: s[x].clone() for x in names} for s in (a, b)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    a["z"].copy_(b["z"]), a["idx"].copy_(b["idx"])
    g.replay()
    torch.cuda.synchronize()
    for x in names:
        assert torch.equal(a[x], want[1][x]), x
    a = state(1)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        step(a, s1), step(b, s2)
    torch.cuda.synchronize()
    for s, w in ((a, want[0]), (b, want[1])):
        for x in names:
            assert torch.equal(s[x], w[x]), x


def test_two_host_threads(ep):
    """Two host threads call the loss at once, each on arrays of its own and
    with a number of experts of its own that the same kernel serves. (The C
    function itself: it runs without the interpreter's lock.)"""
    import sys
    import threading
    got, gate = {}, threading.Barrier(2)

    def calls(e, st):
        z, idx = case(e, 64, e, 4)
        loss, counts = torch.empty(1, device=DEV), torch.empty(1, e, dtype=torch.int32, device=DEV)
        ws = torch.empty(ep.ep_balance_loss_workspace_bytes(64, e), dtype=torch.uint8, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        a = (64, e, 4, 0, z.data_ptr(), idx.data_ptr(), 1, None, 1.0, loss.data_ptr(), counts.data_ptr(), None,
             ws.data_ptr(), ws.numel(), err.data_ptr(), st.cuda_stream)
        torch.cuda.synchronize()
        gate.wait(60)
        failed = sum(ep._lib.ep_balance_loss(*a) != 0 for _ in range(10000))
        st.synchronize()
        l64, c64, _ = ref.balance(z.double(), idx, 0, 1.0, [0, 64])
        got[e] = failed, torch.equal(counts.long(), c64), abs(loss[0].double() - l64).item() <= l64.item() * REL, err.item()
    threads = [threading.Thread(target=calls, args=(e, torch.cuda.Stream())) for e in (68, 128)]
    every = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(every)
    assert got == {68: (0, True, True, 0), 128: (0, True, True, 0)}
