"""ep_linear and ep_expert_linear against the definition in 64 bits.

Tolerances: the bound of moe_ref.linear on the fp32 sums, plus half a step of
the output's type."""
import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ep():
    from combine_top_group_b200 import ep as m
    return m


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def operands(seed, kind, rows, g, cin, cout, act, bias, res):
    r = gen(seed)
    wide, parts = (2 * cout, 2) if act == 3 else (cout, 1)
    s = dict(x_scale=None, w_scale=None)
    x = torch.randn(rows, cin, generator=r, device=DEV)
    w = torch.randn(g, wide, cin, generator=r, device=DEV) * cin ** -0.5
    if kind == "bf16":
        s["x"], s["w"] = x.to(BF), w.to(BF)
    else:
        s["x"], s["w"] = (x * 100).clamp(-448, 448).to(F8), (w * 3000).clamp(-448, 448).to(F8)
        s["x_scale"] = (0.5 + torch.rand(rows, cin // 128, generator=r, device=DEV)) / 100
        s["w_scale"] = (0.5 + torch.rand(g, parts * -(-cout // 128), cin // 128, generator=r, device=DEV)) / 3000
    s["bias"] = torch.randn(g, wide, generator=r, device=DEV) if bias else None
    s["residual"] = torch.randn(rows, cout, generator=r, device=DEV).to(BF) if res else None
    return s


OUT = {"bf16": BF, "fp32": F32, "e4m3": F8}


def outputs(rows, cout, out):
    """out and out_scale, each with 64 canary rows behind."""
    o = torch.full((rows + 64, cout), 7.0, device=DEV).to(OUT[out])
    return o, torch.full((rows + 64, cout // 128), 7.0, device=DEV) if out == "e4m3" else None


def check(s, o, o_scale, at, n, g, act, cout, out):
    """Rows [at, at + n) of the outputs against group g's definition."""
    rows = slice(at, at + n)
    y, err = ref.linear(s["x"][rows], None if s["x_scale"] is None else s["x_scale"][rows], s["w"][g],
                        None if s["w_scale"] is None else s["w_scale"][g],
                        None if s["bias"] is None else s["bias"][g], act,
                        None if s["residual"] is None else s["residual"][rows], cout)
    if out == "e4m3":
        q, scale = ref.quantise(y)
        worst = (err.view(n, -1, 128).amax(2) if n else err.view(n, -1)[:, :0])
        ref.within(o_scale[rows], scale, scale * 1e-5 + worst / 448, "out_scale")
        ref.within(o[rows].float().double() * o_scale[rows].double().repeat_interleave(128, 1), y,
                   ref.e4m3_tolerance(q) * scale.repeat_interleave(128, 1) + err + worst.repeat_interleave(128, 1), "out")
    else:
        half = 2.0 ** -8 if out == "bf16" else 2.0 ** -23
        ref.within(o[rows], y, y.abs() * half + err * (1 + half) + 1e-30, "out")


def untouched(o, o_scale, rows):
    assert (o[rows].float() == 7).all()
    assert o_scale is None or (o_scale[rows] == 7).all()


def dense(ep, kind, rows, cin, cout, act, bias, res, out, seed=1):
    s = operands(seed, kind, rows, 1, cin, cout, act, bias, res)
    o, sc = outputs(rows, cout, out)
    buf = ep.ep_buffer_create(ep.ep_default_config(1, 1, 128, 1, 1), device=DEV)
    ep.ep_linear(buf, s["x"], s["w"], o[:rows], x_scale=s["x_scale"], w_scale=s["w_scale"], bias=s["bias"],
                 residual=s["residual"], act=act, out_scale=None if sc is None else sc[:rows])
    assert ep.ep_check_errors(buf) == 0
    check(s, o, sc, 0, rows, 0, act, cout, out)
    untouched(o, sc, slice(rows, None))


@pytest.mark.parametrize("rows", [1, 2, 15, 17, 32, 33, 64, 65, 127, 129, 200, 257])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("cout", [8, 100, 256, 300])
def test_dense_rows(ep, rows, kind, cout):
    dense(ep, kind, rows, 256, cout, 0, True, False, "bf16")


@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("bias,res", [(False, False), (True, True)])
def test_dense_epilogues(ep, act, kind, out, bias, res):
    for rows, cout in ((3, 128), (150, 384)):
        dense(ep, kind, rows, 384, cout, act, bias, res, out)


@pytest.mark.parametrize("kind,cin", [("bf16", 8), ("bf16", 16), ("bf16", 72), ("bf16", 200), ("bf16", 1000), ("bf16", 4104),
                                      ("e4m3", 128), ("e4m3", 640), ("e4m3", 4224), ("bf16", 7168), ("e4m3", 7168)])
@pytest.mark.parametrize("rows", [1, 40, 140])
def test_dense_depths(ep, kind, cin, rows):
    dense(ep, kind, rows, cin, 192, 1, True, False, "fp32")
    dense(ep, kind, rows, cin, 64, 3, False, True, "bf16")


@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("bias,res", [(False, False), (True, True)])
def test_many_rows(ep, act, kind, out, bias, res):
    """Rows enough for the widest tiles: whole and ragged ones, several to a CTA."""
    for rows, cin, cout in ((256, 128, 256), (385, 384, 384), (1000, 256, 640)):
        dense(ep, kind, rows, cin, cout, act, bias, res, out)


@pytest.mark.parametrize("cout", [129, 250, 260, 264, 500, 516, 1000])
@pytest.mark.parametrize("act", [0, 3])
def test_many_rows_odd_widths(ep, cout, act):
    for out in ("bf16", "fp32"):
        dense(ep, "bf16", 300, 72, cout, act, True, True, out)
    dense(ep, "e4m3", 270, 128, cout, act, True, True, "bf16")


@pytest.mark.parametrize("kind,cin", [("bf16", 8), ("bf16", 1000), ("bf16", 7168), ("e4m3", 128), ("e4m3", 2048), ("e4m3", 7168)])
def test_many_rows_depths(ep, kind, cin):
    """More tiles than pairs of CTAs, so that the ring and the accumulators wrap from tile to tile."""
    dense(ep, kind, 2600, cin, 2048, 0, False, False, "fp32")
    dense(ep, kind, 2600, cin, 1024, 3, True, False, "bf16")


@pytest.mark.parametrize("cout", [1, 2, 3, 5, 7, 9, 31, 63, 65, 127, 129, 191, 255, 257, 511, 1023])
@pytest.mark.parametrize("act", [0, 3])
def test_dense_odd_widths(ep, cout, act):
    """Widths whose rows are not 4- or 8-byte multiples, alone in a call."""
    for out in ("bf16", "fp32"):
        dense(ep, "bf16", 37, 64, cout, act, True, True, out)
    dense(ep, "e4m3", 21, 128, cout, act, True, True, "bf16")


def buffer(ep, R, T, E, K, flags=0, hidden=128):
    cfg = ep.ep_default_config(R, T, hidden, E, K)
    cfg.flags = flags
    return ep.ep_buffer_create(cfg, device=DEV)


def routed(seed, n, e, k, mask=0.1, hot=0.0):
    r = gen(seed)
    z = torch.randn(n, e, generator=r, device=DEV) - hot * torch.log1p(torch.arange(e, device=DEV).float())
    idx = z.topk(k, dim=1).indices.int()
    idx = torch.where(torch.rand(n, k, generator=r, device=DEV) < mask, -1, idx).contiguous()
    return idx, torch.rand(n, k, generator=r, device=DEV)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("R,T,E,K,cin,cout,act,out", [
    (1, 5, 4, 1, 128, 128, 0, "bf16"),          # most experts empty
    (2, 9, 8, 3, 256, 200, 3, "bf16"),
    (1, 1, 64, 2, 128, 72, 1, "fp32"),          # one token, 62 empty experts
    (4, 40, 16, 4, 384, 256, 3, "e4m3"),
    (2, 300, 6, 2, 128, 136, 2, "bf16"),        # several tiles per expert
    (1, 700, 2, 1, 256, 384, 0, "e4m3"),
    (8, 16, 256, 8, 128, 128, 3, "bf16"),
    (1, 4000, 5, 2, 128, 256, 3, "e4m3"),       # many rows per expert, unevenly
    (2, 1500, 6, 3, 256, 300, 0, "bf16"),
    (1, 64, 1024, 4, 128, 64, 0, "fp32"),       # the most experts
])
def test_experts(ep, kind, R, T, E, K, cin, cout, act, out):
    buf = buffer(ep, R, T, E, K)
    idx, wt = routed(T, R * T, E, K, hot=0.8)
    ep.ep_get_layout(buf, T, topk_idx=idx, topk_w=wt)
    rows = R * T * K
    s = operands(2, kind, rows, E, cin, cout, act, True, True)
    off = ep.ep_buffer_layout(buf, T)["expert_off"].tolist()
    # rows behind the last filled one are read by tiles, but reach no output
    if kind == "bf16":
        s["x"][off[-1]:] = float("nan")
    else:
        s["x_scale"][off[-1]:] = float("nan")
    o, sc = outputs(rows, cout, out)
    ep.ep_expert_linear(buf, T, s["x"], s["w"], o, x_scale=s["x_scale"], w_scale=s["w_scale"], bias=s["bias"],
                        residual=s["residual"], act=act, out_scale=sc)
    assert ep.ep_check_errors(buf) == 0
    for g in range(E):
        check(s, o, sc, off[g], off[g + 1] - off[g], g, act, cout, out)
    untouched(o, sc, slice(off[-1], None))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_row_stays_apart(ep, bad):
    """A row with NaN or infinity spoils that row of the outputs alone, and an
    expert's weights spoil that expert's rows alone."""
    T, E, cin, cout = 90, 3, 128, 128
    buf = buffer(ep, 1, T, E, 1)
    idx = (torch.arange(T, device=DEV, dtype=torch.int32) * E // T).view(T, 1).contiguous()
    ep.ep_get_layout(buf, T, topk_idx=idx, topk_w=torch.ones(T, 1, device=DEV))
    s = operands(3, "bf16", T, E, cin, cout, 0, False, False)
    s["x"][31, 5] = bad   # expert 1's second row
    s["w"][2, 7, 9] = bad
    o, _ = outputs(T, cout, "bf16")
    ep.ep_expert_linear(buf, T, s["x"], s["w"], o)
    fine = o[:T].isfinite()
    want = torch.ones_like(fine)
    want[31] = False
    want[60:, 7] = False
    assert torch.equal(fine, want)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("R,T,E,K", [(2, 12, 8, 2), (4, 33, 4, 2), (8, 16, 64, 6), (2, 900, 4, 2), (1, 1500, 2, 1)])
def test_low_latency_regions(ep, kind, R, T, E, K):
    buf = buffer(ep, R, T + 3, E, K, ep.EP_FLAG_LOW_LATENCY)
    idx, wt = routed(1, R * T, E, K, hot=0.5)
    ep.ep_get_layout(buf, T, topk_idx=idx, topk_w=wt)
    cnt = ep.ep_buffer_layout(buf, T)["cnt"].tolist()
    rows, region = E * R * (T + 3), T + 3
    s = operands(4, kind, rows, E, 256, 192, 3, True, False)
    o, sc = outputs(rows, 192, "bf16")
    ep.ep_expert_linear(buf, T, s["x"], s["w"], o, x_scale=s["x_scale"], w_scale=s["w_scale"], bias=s["bias"], act=3)
    assert ep.ep_check_errors(buf) == 0
    for e in range(E):
        for r in range(R):
            at, n = (e * R + r) * region, cnt[r][e]
            check(s, o, sc, at, n, e, 3, 192, "bf16")
            untouched(o, sc, slice(at + n, at + region))


def test_dedup_rows(ep):
    """The rows that the local permutation of a deduplicated receive lays out."""
    R, T, E, K, H, cout = 2, 30, 8, 3, 256, 128
    buf = buffer(ep, R, T, E, K, ep.EP_FLAG_DEDUP, H)
    idx, wt = routed(9, R * T, E, K)
    ep.ep_get_layout(buf, T, topk_idx=idx, topk_w=wt)
    ep.ep_dispatch_dedup(buf, T, torch.randn(R * T, H, generator=gen(1), device=DEV).to(BF))
    ep.ep_permute(buf, T)
    x = ep.ep_buffer_recv(buf)["recv_x"]
    s = dict(operands(5, "bf16", 1, E, H, cout, 1, True, False), x=x)
    o, _ = outputs(R * T * K, cout, "bf16")
    ep.ep_expert_linear(buf, T, x, s["w"], o, bias=s["bias"], act=1)
    assert ep.ep_check_errors(buf) == 0
    off = ep.ep_buffer_layout(buf, T)["expert_off"].tolist()
    for g in range(E):
        check(s, o, None, off[g], off[g + 1] - off[g], g, 1, cout, "bf16")
    untouched(o, None, slice(off[-1], None))


def test_large_calls_on_two_streams(ep):
    """Calls that each take every SM, with pairs and with clusters, at once."""
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    sets = []
    for seed, (rows, cin, cout, st) in enumerate(((3000, 1024, 4096, s1), (40, 8192, 2048, s2), (700, 2048, 512, s1), (300, 4096, 1024, s2))):
        s = operands(seed, "bf16", rows, 1, cin, cout, 0, False, False)
        want, got = torch.empty(rows, cout, dtype=BF, device=DEV), torch.empty(rows, cout, dtype=BF, device=DEV)
        sets.append((buffer(ep, 1, 1, 1, 1), s, want, got, st))
    for buf, s, want, _, _ in sets:
        ep.ep_linear(buf, s["x"], s["w"], want)
    torch.cuda.synchronize()
    for _ in range(20):
        for buf, s, _, got, st in sets:
            ep.ep_linear(buf, s["x"], s["w"], got, stream=st)
    torch.cuda.synchronize()
    for buf, _, want, got, _ in sets:
        assert torch.equal(want, got) and ep.ep_check_errors(buf) == 0


@pytest.mark.parametrize("rank", [0, 3])
def test_shard(ep, rank):
    """A shard's own experts on the rows that all ranks send it."""
    R, T, E, K, cin, cout = 4, 50, 16, 3, 128, 128
    one = buffer(ep, R, T, E, K)
    idx, wt = routed(6, R * T, E, K)
    ep.ep_get_layout(one, T, topk_idx=idx, topk_w=wt)
    cnt = ep.ep_buffer_layout(one, T)["cnt"].clone()
    buf = buffer(ep, R, T, E, K, ep.EP_FLAG_SHARD)
    ep.ep_shard_layout(buf, rank, T, topk_idx=idx[rank * T:(rank + 1) * T].contiguous(),
                       topk_w=wt[rank * T:(rank + 1) * T].contiguous())
    rows, L = R * T * K, E // R
    s = operands(5, "bf16", rows, L, cin, cout, 3, False, False)
    o, sc = outputs(rows, cout, "bf16")
    with pytest.raises(ep.EpError):
        ep.ep_expert_linear(buf, T, s["x"], s["w"], o, act=3)
    ep.ep_buffer_shard(buf, T)["cnt_all"].copy_(cnt)
    ep.ep_shard_place(buf, rank, T)
    ep.ep_expert_linear(buf, T, s["x"], s["w"], o, act=3)
    assert ep.ep_check_errors(buf) == 0
    off = ep.ep_buffer_shard(buf, T)["recv_off"].tolist()
    assert off[-1] == int(cnt[:, rank * L:(rank + 1) * L].sum())
    for g in range(L):
        check(s, o, sc, off[g], off[g + 1] - off[g], g, 3, cout, "bf16")
    untouched(o, sc, slice(off[-1], None))


@pytest.mark.parametrize("T,bad", [(30, {3: 1000}), (30, {2: -7}), (30, {1: 50, 2: 20}), (2000, {4: 2 ** 30})])
def test_bad_offsets(ep, T, bad):
    """Row offsets that leave the array are reported and reach no memory
    outside it; the other experts' rows come out as they should."""
    E, cin, cout = 4, 128, 256
    buf = buffer(ep, 1, T, E, 1)
    idx = (torch.arange(T, device=DEV, dtype=torch.int32) * E // T).view(T, 1).contiguous()
    ep.ep_get_layout(buf, T, topk_idx=idx, topk_w=torch.ones(T, 1, device=DEV))
    off = ep.ep_buffer_layout(buf, T)["expert_off"]
    for i, v in bad.items():
        off[i] = v
    now = off.tolist()
    s = operands(3, "bf16", T, E, cin, cout, 0, False, False)
    o, _ = outputs(T, cout, "bf16")
    ep.ep_expert_linear(buf, T, s["x"], s["w"], o)
    wrong = [g for g in range(E) if now[g + 1] > now[g] and (now[g] < 0 or now[g + 1] > T)]
    assert ep.ep_check_errors(buf) == (ep.EP_DEVERR_ROW_BOUNDS if wrong else 0)
    kept = [g for g in range(E) if 0 <= now[g] < now[g + 1] <= T]
    spans = [(now[g], now[g + 1]) for g in kept]
    for g, (a, b) in zip(kept, spans):
        if not any(c < b and a < d for c, d in spans if (c, d) != (a, b)):
            check(s, o, None, a, b - a, g, 0, cout, "bf16")
    covered = torch.zeros(T + 64, dtype=torch.bool)
    for a, b in spans:
        covered[a:b] = True
    untouched(o, None, (~covered).to(DEV))


def test_residual_in_place(ep):
    rows, cin, cout = 70, 192, 100
    s = operands(7, "bf16", rows, 1, cin, cout, 2, True, True)
    buf = buffer(ep, 1, 1, 1, 1)
    o, _ = outputs(rows, cout, "bf16")
    ep.ep_linear(buf, s["x"], s["w"], o[:rows], bias=s["bias"], residual=s["residual"], act=2)
    ep.ep_linear(buf, s["x"], s["w"], s["residual"], bias=s["bias"], residual=s["residual"], act=2)
    assert torch.equal(o[:rows], s["residual"])


def test_no_rows(ep):
    buf = buffer(ep, 1, 8, 4, 2)
    s = operands(7, "bf16", 16, 4, 64, 64, 0, False, False)
    o, _ = outputs(16, 64, "bf16")
    ep.ep_linear(buf, s["x"][:0], s["w"][:1], o[:0])
    ep.ep_get_layout(buf, 0, logits=torch.zeros(1, 4, device=DEV))
    ep.ep_expert_linear(buf, 0, s["x"], s["w"], o)
    ep.ep_get_layout(buf, 8, topk_idx=torch.full((8, 2), -1, dtype=torch.int32, device=DEV), topk_w=torch.zeros(8, 2, device=DEV))
    ep.ep_expert_linear(buf, 8, s["x"], s["w"], o)
    assert ep.ep_check_errors(buf) == 0
    untouched(o, None, slice(None))


def test_offsets_past_32_bits(ep):
    """The last rows of an x, and the last expert of weights, of more than 2^31
    values."""
    rows, cin, cout = 2 ** 31 // 4096 + 5, 4096, 8
    buf = buffer(ep, 1, 1, 1, 1)
    x = torch.zeros(rows, cin, dtype=BF, device=DEV)
    x[-3:] = torch.randn(3, cin, generator=gen(1), device=DEV).to(BF)
    s = operands(1, "bf16", 1, 1, cin, cout, 0, False, False)
    o, _ = outputs(rows, cout, "bf16")
    ep.ep_linear(buf, x, s["w"], o[:rows])
    s["x"] = x
    check(s, o, None, rows - 3, 3, 0, 0, cout, "bf16")
    untouched(o, None, slice(rows, None))
    del x
    E, cin, cout = 33, 8192, 8192
    w = torch.zeros(E, cout, cin, dtype=BF, device=DEV)
    w[-1] = torch.randn(cout, cin, generator=gen(2), device=DEV).to(BF)
    buf = buffer(ep, 1, 4, E, 1)
    ep.ep_get_layout(buf, 4, topk_idx=torch.full((4, 1), E - 1, dtype=torch.int32, device=DEV), topk_w=torch.ones(4, 1, device=DEV))
    s = dict(x=torch.randn(4, cin, generator=gen(3), device=DEV).to(BF), x_scale=None, w=w, w_scale=None, bias=None, residual=None)
    o, _ = outputs(4, cout, "bf16")
    ep.ep_expert_linear(buf, 4, s["x"], w, o)
    check(s, o, None, 0, 4, E - 1, 0, cout, "bf16")


def test_refusals(ep):
    buf = buffer(ep, 1, 8, 4, 2)
    idx, wt = routed(1, 8, 4, 2, 0)
    ep.ep_get_layout(buf, 8, topk_idx=idx, topk_w=wt)
    a = operands(1, "bf16", 16, 4, 64, 128, 0, True, True)
    f = operands(1, "e4m3", 16, 4, 128, 128, 0, False, False)
    o, q = torch.empty(16, 128, dtype=BF, device=DEV), torch.empty(16, 128, dtype=F8, device=DEV)
    sc = torch.empty(16, 1, device=DEV)

    def refuses(status, *args, **kw):
        with pytest.raises(ep.EpError) as e:
            ep.ep_expert_linear(buf, *args, **kw)
        assert e.value.status == status and str(e.value)
    x, w = a["x"], a["w"]
    refuses(1, 7, x, w, o)                                   # not the last layout's T
    refuses(1, 8, x[:15], w, o)                              # too few rows
    refuses(1, 8, x, w[:3], o)                               # too few experts
    refuses(1, 8, x, w, o[:, :64])                           # not contiguous
    refuses(1, 8, x, w, o, act=9)
    refuses(1, 8, x, w, o, act=3)                            # no up rows
    refuses(1, 8, x, w, q)                                   # e4m3 out without scales
    refuses(1, 8, x, w, o, out_scale=sc)
    refuses(1, 8, x.half(), w, o)
    refuses(1, 8, x.cpu(), w, o)
    refuses(1, 8, x, f["w"], o)                              # mixed types
    refuses(1, 8, f["x"], f["w"], o)                         # e4m3 without scales
    refuses(1, 8, f["x"], f["w"], o, x_scale=f["x_scale"])
    refuses(1, 8, x, w, o, bias=a["bias"][:, :64].contiguous())
    refuses(1, 8, x, w, o, residual=a["residual"].float())
    refuses(5, 8, x[:, :60].contiguous(), w[:, :, :60].contiguous(), o)      # in_features % 8
    refuses(5, 8, x, w[:, :64].contiguous(), q[:, :64].contiguous(), out_scale=sc[:, :0].contiguous())
    flat = torch.empty(16 * 64 + 8, dtype=BF, device=DEV)
    refuses(1, 8, flat[4:4 + 16 * 64].view(16, 64), w, o)    # 8-byte aligned rows
    assert ep.ep_check_errors(buf) == 0


def test_graph_and_streams(ep):
    """A captured call replays on new routing and new rows; calls on two
    streams with a buffer each give the bits of plain ones."""
    T, E, K, cin, cout = 64, 8, 2, 256, 256

    def state(seed):
        buf = buffer(ep, 1, T, E, K)
        idx, wt = routed(seed, T, E, K, 0.1, 1.0)
        s = operands(seed, "bf16", T * K, E, cin, cout, 3, True, False)
        return dict(buf=buf, idx=idx, wt=wt, o=torch.zeros(T * K, cout, dtype=BF, device=DEV), **s)

    def step(s, st=None):
        ep.ep_get_layout(s["buf"], T, topk_idx=s["idx"], topk_w=s["wt"], stream=st)
        ep.ep_expert_linear(s["buf"], T, s["x"], s["w"], s["o"], bias=s["bias"], act=3, stream=st)
    a, b = state(1), state(2)
    step(a), step(b)
    want = a["o"].clone(), b["o"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    for k in ("idx", "wt", "x", "w", "bias"):
        a[k].copy_(b[k])
    a["o"].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a["o"], want[1])
    a = state(1)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        step(a, s1), step(b, s2)
    torch.cuda.synchronize()
    assert torch.equal(a["o"], want[0]) and torch.equal(b["o"], want[1])
    assert ep.ep_check_errors(a["buf"]) == 0 and ep.ep_check_errors(b["buf"]) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_moe_block(ep, fp8):
    """The block as a model runs it: norm, router projection, routing, dispatch,
    the experts' two layers, combine onto the residual stream, and the router's
    loss with its gradient; against the same steps in 64 bits on the kernels' routing."""
    N, H, I, E, K = 96, 512, 256, 8, 2
    r = gen(1)
    x, res = (torch.randn(N, H, generator=r, device=DEV).to(BF) for _ in range(2))
    gamma = 1 + 0.1 * torch.randn(H, generator=r, device=DEV)
    wr = (torch.randn(1, E, H, generator=r, device=DEV) * H ** -0.5).to(BF)
    kind = "e4m3" if fp8 else "bf16"
    up, down = operands(2, kind, 1, E, H, I, 3, True, False), operands(3, kind, 1, E, I, H, 0, False, False)
    cfg = ep.ep_default_config(1, N, H, E, K)
    cfg.flags = ep.EP_FLAG_FP8 if fp8 else 0
    buf = ep.ep_buffer_create(cfg, device=DEV)
    h, y, logits = torch.empty_like(x), torch.empty_like(x), torch.empty(N, E, device=DEV)
    ep.ep_rmsnorm(x, gamma, 1e-6, residual=res, h=h, y=y)
    ep.ep_linear(buf, y, wr, logits)
    ep.ep_get_layout(buf, N, logits=logits, route=ep.EP_ROUTE_SOFTMAX_RENORM)
    ep.ep_dispatch(buf, N, y)
    recv, lay = ep.ep_buffer_recv(buf), ep.ep_buffer_layout(buf, N)
    z = torch.empty(N * K, I, dtype=F8 if fp8 else BF, device=DEV)
    zs = torch.empty(N * K, I // 128, device=DEV) if fp8 else None
    ep.ep_expert_linear(buf, N, recv["recv_x"], up["w"], z, x_scale=recv["recv_scale"], w_scale=up["w_scale"],
                        bias=up["bias"], act=ep.EP_ACT_SWIGLU, out_scale=zs)
    out_rows = torch.empty(N * K, H, dtype=BF, device=DEV)
    ep.ep_expert_linear(buf, N, z, down["w"], out_rows, x_scale=zs, w_scale=down["w_scale"])
    out = torch.empty_like(x)
    ep.ep_combine(buf, N, out_rows, None, out)
    loss, counts = torch.empty(1, device=DEV), torch.empty(1, E, dtype=torch.int32, device=DEV)
    ws = torch.empty(ep.ep_balance_loss_workspace_bytes(N, E, 1), dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dl = torch.empty_like(logits)
    ep.ep_balance_loss(logits, lay["topk_idx"], ep.EP_SCORE_SOFTMAX, 0.01, loss, counts, ws, err)
    ep.ep_balance_loss_backward(logits, counts, K, ep.EP_SCORE_SOFTMAX, 0.01, dl)
    assert ep.ep_check_errors(buf) == 0 and err.item() == 0
    # the same in 64 bits, expert by expert, on the kernels' top-k
    _, _, n64 = ref.norm(x, res, gamma, 1e-6)
    l64 = n64 @ wr[0].double().t()
    idx, w = lay["topk_idx"].long(), lay["topk_w"].double()
    want = torch.zeros(N, H, dtype=torch.float64, device=DEV)
    w_up, w_down = ref.weight64(up["w"], up["w_scale"], I), ref.weight64(down["w"], down["w_scale"], H)
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        a = n64[t] @ w_up[e].t() + up["bias"][e].double()
        b = (torch.nn.functional.silu(a[:, :I]) * a[:, I:]) @ w_down[e].t()
        want.index_add_(0, t, w[t, k][:, None] * b)
    # bf16 (2^-8) or e4m3 (2^-4) roundings of the rows, the hidden values and the outputs, independent over H and I values
    rel = ((out.double() - want).norm() / want.norm()).item()
    assert rel < (2.0 ** -4 if fp8 else 2.0 ** -7), rel
    ref.within(logits, l64, n64.abs() @ wr[0].double().abs().t() * 2.0 ** -8, "logits")
    b64 = ref.balance(logits.double(), lay["topk_idx"], 0, 0.01, [0, N])
    assert torch.equal(counts.long(), b64[1]) and torch.equal(counts[0], lay["num_tokens_per_expert"])
    assert abs(loss[0].double() - b64[0]) <= b64[0] * 2.0 ** -17
    assert dl.isfinite().all()


def test_rows_up_to_2_31(ep):
    """The most rows that a call takes: the tile count of 2^31 - 1 rows needs
    more than 31 bits on its way."""
    rows, cin = 2 ** 31 - 1, 8
    x = torch.zeros(rows, cin, dtype=BF, device=DEV)
    x[-3:] = torch.randn(3, cin, generator=gen(1), device=DEV).to(BF)
    s = operands(1, "bf16", 1, 1, cin, 1, 0, False, False)
    o = torch.full((rows, 1), 7.0, dtype=BF, device=DEV)
    buf = buffer(ep, 1, 1, 1, 1)
    ep.ep_linear(buf, x, s["w"], o)
    assert ep.ep_check_errors(buf) == 0
    s["x"] = x
    check(s, o, None, rows - 3, 3, 0, 0, 1, "bf16")
    assert not o[:-3].any()


def test_offsets_too_far_apart(ep):
    """An expert whose offsets are more than 2^31 apart is reported too."""
    T, E, cin, cout = 30, 4, 128, 256
    buf = buffer(ep, 1, T, E, 1)
    idx = (torch.arange(T, device=DEV, dtype=torch.int32) * E // T).view(T, 1).contiguous()
    ep.ep_get_layout(buf, T, topk_idx=idx, topk_w=torch.ones(T, 1, device=DEV))
    off = ep.ep_buffer_layout(buf, T)["expert_off"]
    off[3], off[4] = -2, 2 ** 31 - 1
    now = off.tolist()
    s = operands(3, "bf16", T, E, cin, cout, 0, False, False)
    o, _ = outputs(T, cout, "bf16")
    ep.ep_expert_linear(buf, T, s["x"], s["w"], o)
    assert ep.ep_check_errors(buf) == ep.EP_DEVERR_ROW_BOUNDS
    for g in range(2):
        check(s, o, None, now[g], now[g + 1] - now[g], g, 0, cout, "bf16")
    untouched(o, None, slice(now[2], None))


@pytest.mark.parametrize("flags", [0, 2, 4])
def test_no_layout_yet(ep, flags):
    """Before any layout every T is refused, the negative ones as well."""
    buf = buffer(ep, 1, 8, 4, 2, flags)
    s = operands(7, "bf16", 64, 4, 128, 64, 0, False, False)
    o, _ = outputs(64, 64, "bf16")
    y = torch.zeros(64, 128, dtype=BF, device=DEV)
    calls = [lambda t: ep.ep_expert_linear(buf, t, s["x"], s["w"], o)]
    calls += [lambda t: ep.ep_dispatch_dedup(buf, t, y), lambda t: ep.ep_permute(buf, t)] if flags == 4 else \
        [lambda t: ep.ep_dispatch(buf, t, y), lambda t: ep.ep_combine(buf, t, y, None, y.clone())]
    for call in calls:
        for t in (-1, 0, 8):
            with pytest.raises(ep.EpError) as e:
                call(t)
            assert e.value.status == ep.EP_ERR_INVALID
    untouched(o, None, slice(None))


def positive(seed, kind, rows, cin, cout):
    """Operands of one sign, so that nothing cancels, rows of sizes spread over an octave."""
    s = operands(seed, kind, rows, 1, cin, cout, 0, False, False)
    spread = 1 + torch.rand(rows, 1, generator=gen(seed + 1), device=DEV)
    s["w"] = s["w"].float().abs().to(s["w"].dtype)
    s["x"] = (s["x"].float().abs() * (spread if kind == "bf16" else 1)).to(s["x"].dtype)
    return s


def product(s, cout):
    x = s["x"].double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double().repeat_interleave(128, 1)
    w = ref.weight64(s["w"], s["w_scale"], cout)[0]
    return torch.cat([x @ w[n:n + 1024].t() for n in range(0, cout, 1024)], 1)


# rows, out_features: a cluster for each tile; one CTA for each; a cluster for 128 rows; pairs of CTAs
KERNELS = [(3, 512), (40, 148 * 512), (512, 2048), (2048, 2048)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,cout", KERNELS)
def test_exactness_of_deep_sums(ep, kind, rows, cout):
    """fp32 outputs of 7168 channels. Tensor memory cuts its sums. bf16: 32
    steps of 16 channels at a time (8e-7 in the mean, with little spread), then 14
    parts and at most 8 of a cluster are added in fp32 (2^-24 each at most, of
    either sign: under 1e-6). All 448 steps in one go cut 2.7e-5. e4m3: 56 blocks
    of 4 steps, each scaled and added in fp32, with 72 roundings of 2^-24 at most."""
    s = positive(1, kind, rows, 7168, cout)
    o = torch.empty(rows, cout, device=DEV)
    ep.ep_linear(buffer(ep, 1, 1, 1, 1), s["x"], s["w"], o, x_scale=s["x_scale"], w_scale=s["w_scale"])
    y = product(s, cout)
    ref.within(o, y, y * (2e-6 if kind == "bf16" else 72 * 2.0 ** -24), "out")


@pytest.mark.parametrize("rows,cout,cin", [(3, 128, 2 ** 19), (300, 256, 2 ** 19), (4096, 2048, 2 ** 15)])
def test_bf16_outputs_of_the_deepest_sums(ep, rows, cout, cin):
    """bf16 out: half a step of the value itself, and what the sum may lose:
    128 steps in tensor memory (5e-6), 256 parts added in fp32 (2^-24 each at
    most). In one go 2^15 channels lose 1.7e-4, and one output in 30 is rounded
    the wrong way."""
    s = positive(1, "bf16", rows, cin, cout)
    o = torch.empty(rows, cout, dtype=BF, device=DEV)
    ep.ep_linear(buffer(ep, 1, 1, 1, 1), s["x"], s["w"], o)
    y = product(s, cout)
    half = torch.ldexp(torch.ones_like(y), torch.frexp(y).exponent - 9)
    ref.within(o, y, half + y * 2e-5, "out")


def test_waits_give_up(ep):
    """The kernels' waits end after their limit, or when another warp has given
    up, and the next call on the same context works."""
    import time
    words = torch.zeros(4, dtype=torch.int32, device=DEV)
    t0 = time.perf_counter()
    bits = ep.ep_selftest_wait_timeout(words, 50_000_000)
    assert bits & ep.EP_DEVERR_TIMEOUT
    assert words[0] == 1 and words[3] == 1
    # three waits of 50 ms; the linear layers' run on the SM's clock, up to 2 GHz; none took its full 2 s
    assert 0.14 < time.perf_counter() - t0 < 1.5
    dense(ep, "bf16", 70, 256, 300, 0, True, False, "bf16")
