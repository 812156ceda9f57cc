"""The block boundary (norms, gate, residual) and its gradients through the
ABI, against the definitions in 64 bits.

Bounds, fixed before any run, with u = 2^-24:
  - a bf16 output is rounded once: half a unit in its last place is 2^-9 of
    its size, and 2^-8 leaves room for the fp32 value before it;
  - fp32 values of a row: sums over h terms with at most 3 + log2(threads)
    roundings a path beside the NV * 8 terms of a thread, statistics that
    enter twice, and the cancellations of x + z and of the gradient's
    projections: 64 u of the row's largest magnitude of the terms;
  - a column sum over M rows: (M + 64) u times the sum of its terms'
    magnitudes, the bound of a sum in any order plus 64 u a term."""
import pytest
import torch

import ops_ref as ref

U = 2.0 ** -24
BF, F32, D = torch.bfloat16, torch.float32, torch.float64


def close_row(got, want, scale, what):
    """|got - want| within the rounding of got's type and 64 u of `scale` (per row)."""
    got = got.detach().cpu()
    unit = 2.0 ** -8 if got.dtype == BF else 2.0 ** -23
    err = (got.to(D) - want).abs()
    lim = unit * want.abs() + 64 * U * scale
    assert torch.isfinite(got.to(D)).all(), f"{what}: not finite"
    assert (err <= lim).all(), f"{what}: {float((err / lim.clamp_min(1e-300)).max()):.3g} times the bound"


def close_sum(got, want, terms, M, what):
    got = got.detach().cpu()
    unit = 2.0 ** -8 if got.dtype == BF else 2.0 ** -23
    err, lim = (got.to(D) - want).abs(), unit * want.abs() + (M + 64) * U * terms
    assert (err <= lim + 1e-30).all(), f"{what}: {float((err / lim.clamp_min(1e-300)).max()):.3g} times the bound"


def make(M, h, post, pre, gate, res, seed=0, bias=True, weights=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, z = (2 * rnd(M, h)).to(res), (rnd(M, h) + 0.5).to(BF)
    dn, dy = rnd(M, h).to(BF), rnd(M, h).to(res)
    vec = lambda on, c, s: (c + s * rnd(h)).to(BF) if on else None  # noqa: E731
    d = dict(post=post, pre=pre, alpha=0.75, eps=1e-5,
             w_post=vec(weights and post != "none", 1, 0.2), b_post=vec(bias and post == "layer", 0, 0.2),
             w_pre=vec(weights and pre != "none", 1, 0.2), b_pre=vec(bias and pre == "layer", 0, 0.2),
             gate=rnd(gate, h).to(BF) if gate else None)
    return x, z, dn, dy, d


def wide(d):
    return {k: v.to(D) if torch.is_tensor(v) else v for k, v in d.items()}


def shards(t, p):
    return None if t is None else [c.contiguous().cuda() for c in t.chunk(p)] if t.shape[0] else [t.clone().cuda() for _ in range(p)]


def call_args(tp, d):
    kind = {"none": tp.TP_NORM_NONE, "rms": tp.TP_NORM_RMS, "layer": tp.TP_NORM_LAYER}
    a = {k: v.cuda() if torch.is_tensor(v) else v for k, v in d.items()}
    a["post"], a["pre"] = kind[d["post"]], kind[d["pre"]]
    return a


def cat(ts):
    return torch.cat([t.cpu() for t in ts])


def nan_like(ts, dtype=None):
    return [torch.full_like(t, float("nan"), dtype=dtype) for t in ts]


def check_fwd(tp, p, M, h, post, pre, gate, res, has_z=True, has_n=True, **kw):
    x, z, _, _, d = make(M, h, post, pre, gate, res, **kw)
    if not has_z:
        z = None
    xs, zs = shards(x, p), shards(z, p)
    ys = nan_like(xs) if has_z else None
    ns = nan_like(xs, BF) if has_n else None
    tp.tp_block_norm_fwd(xs, zs, ys, ns, **call_args(tp, d))
    y, n = ref.block_fwd(x.to(D), None if z is None else z.to(D), wide(d))
    part = x.to(D).abs() + (y - x.to(D)).abs()
    if has_z:
        close_row(cat(ys), y, part.amax(1, keepdim=True), "y")
    if has_n:
        w = 1 if d["w_pre"] is None else d["w_pre"].to(D).abs()
        dev = 1 / ref.hat(y, pre, d["eps"])[1]
        close_row(cat(ns), n, (part.amax(1, keepdim=True) / dev + 1) * w + 1, "n")


def check_bwd(tp, p, M, h, post, pre, gate, res, out=F32, has_z=True, has_dn=True, has_dy=True, **kw):
    y, z, dn, dy, d = make(M, h, post, pre, gate, res, **kw)
    if not has_z:
        z, d["gate"], d["post"], d["w_post"], d["b_post"] = None, None, "none", None, None
    if not has_dn:
        dn, d["pre"], d["w_pre"], d["b_pre"] = None, "none", None, None
    if not has_dy:
        dy = None
    post, pre = d["post"], d["pre"]
    ys, zs, dns, dys = shards(y, p), shards(z, p), shards(dn, p), shards(dy, p)
    dx, dz = nan_like(ys), nan_like(ys, BF) if has_z else None
    names = {"dw_post": (h,), "db_post": (h,), "dw_pre": (h,), "db_pre": (h,), "dgate": (gate, h)}
    have = {"dw_post": post != "none", "db_post": post == "layer", "dw_pre": pre != "none", "db_pre": pre == "layer",
            "dgate": d["gate"] is not None}
    grads = {k: torch.full(s, float("nan"), dtype=out, device="cuda") if have[k] else None for k, s in names.items()}
    ws = tp.workspace(tp.TP_OP_BLOCK_NORM_BWD, p, M, h, 0)
    ws.fill_(0xFF)  # need not be zero-filled
    tp.tp_block_norm_bwd(zs, ys if has_dn else None, dns, dys, dx, dz, ws, **grads, **call_args(tp, d))
    want = ref.block_bwd(y.to(D), None if z is None else z.to(D), None if dn is None else dn.to(D),
                         None if dy is None else dy.to(D), wide(d))
    size = torch.zeros((M, 1), dtype=D) if dy is None else dy.to(D).abs().amax(1, keepdim=True)
    if has_dn:
        hy, ry = ref.hat(y.to(D), pre, d["eps"])
        u = dn.to(D).abs() * (1 if d["w_pre"] is None else d["w_pre"].to(D).abs())
        size = size + ry * u.amax(1, keepdim=True) * (2 + hy.abs().amax(1, keepdim=True) ** 2)
    close_row(cat(dx), want["dx"], size, "dx")
    if has_z:
        hz, rz = ref.hat(z.to(D), post, d["eps"])
        q = torch.ones((M, h), dtype=D)
        for k in ("w_post",):
            q = q if d[k] is None else q * d[k].to(D).abs()
        if d["gate"] is not None:
            q = q * ref.rows_of_gate(d["gate"].to(D).abs(), M)
        most = hz.abs().amax(1, keepdim=True) if post != "none" else 0 * rz
        close_row(cat(dz), want["dz"], rz * size * q.amax(1, keepdim=True) * (2 + most ** 2), "dz")
    for k, g in grads.items():
        if g is not None:
            extra = 0.0
            if k in ("dw_post", "db_post", "dgate"):  # their terms hold dx, whose own error is `size`
                s = size * (hz.abs() + 1) * (1 if d["gate"] is None or k == "dgate" else ref.rows_of_gate(d["gate"].to(D).abs(), M))
                if k == "dgate":
                    s = s * (1 if d["w_post"] is None else d["w_post"].to(D).abs()) + size
                    extra = s.view(gate, -1, h).sum(1)
                else:
                    extra = s.sum(0)
            close_sum(g, want[k], want["|" + k + "|"] + extra, M, k)


@pytest.fixture(scope="module")
def tp():
    import gemm_reduce_fusion_gb300 as tp
    return tp


# h: one vector, part of a warp, whole warps, both warp widths, CTAs of odd and
# whole sizes up to the largest; M: one row, fewer rows than workers, ragged
FWD = [(1, 1, 8), (2, 6, 64), (1, 5, 264), (3, 33, 512), (1, 9, 520), (4, 64, 1024), (1, 7, 1032), (2, 4, 2056), (8, 16, 4096),
       (1, 3, 6152), (1, 2, 12288), (1, 2, 16384), (1, 700, 1160), (8, 3000, 72)]


@pytest.mark.gpu
@pytest.mark.parametrize("res", [BF, F32])
@pytest.mark.parametrize("p,M,h", FWD)
def test_forward(tp, p, M, h, res):
    check_fwd(tp, p, M, h, "rms", "rms", 1, res)
    check_fwd(tp, p, M, h, "layer", "layer", M, res)
    check_fwd(tp, p, M, h, "none", "layer", p, res)
    check_fwd(tp, p, M, h, "layer", "rms", 0, res, weights=False)


@pytest.mark.gpu
@pytest.mark.parametrize("res", [BF, F32])
@pytest.mark.parametrize("h", [200, 1160, 4096])
def test_forward_of_one_norm_alone(tp, h, res):
    check_fwd(tp, 2, 10, h, "none", "rms", 0, res, has_z=False)
    check_fwd(tp, 1, 10, h, "none", "layer", 0, res, has_z=False)
    check_fwd(tp, 2, 10, h, "rms", "none", 2, res, has_n=False)
    check_fwd(tp, 1, 10, h, "none", "none", 0, res, has_n=False)


@pytest.mark.gpu
@pytest.mark.parametrize("res,out", [(BF, F32), (F32, F32), (BF, BF)])
@pytest.mark.parametrize("p,M,h", FWD)
def test_backward(tp, p, M, h, res, out):
    check_bwd(tp, p, M, h, "rms", "rms", 1, res, out)
    check_bwd(tp, p, M, h, "layer", "layer", M, res, out)
    check_bwd(tp, p, M, h, "none", "layer", p, res, out)
    check_bwd(tp, p, M, h, "layer", "rms", 0, res, out, weights=False)


@pytest.mark.gpu
@pytest.mark.parametrize("h", [200, 1160, 4096])
def test_backward_without_some_inputs(tp, h):
    check_bwd(tp, 2, 10, h, "none", "rms", 0, BF, has_z=False)
    check_bwd(tp, 2, 10, h, "none", "layer", 0, F32, has_z=False, has_dy=False)
    check_bwd(tp, 1, 10, h, "rms", "none", 5, BF, has_dn=False)
    check_bwd(tp, 1, 10, h, "layer", "rms", 1, BF, has_dy=False)


@pytest.mark.gpu
@pytest.mark.parametrize("groups", [2, 3, 7, 100, 350, 700, 2100])
@pytest.mark.parametrize("h", [136, 1160])
def test_gate_groups_that_end_inside_and_between_workers(tp, h, groups):
    check_bwd(tp, 1, 2100, h, "rms", "rms", groups, BF)


@pytest.mark.gpu
def test_a_row_with_nan_or_infinity_keeps_to_itself(tp):
    M, h = 37, 1160
    x, z, dn, dy, d = make(M, h, "layer", "rms", 1, BF)
    a = call_args(tp, d)
    out = []
    for broken in (False, True):
        xb, zb = x.clone(), z.clone()
        if broken:
            xb[5, 7], zb[9, 3], zb[20, 0] = float("nan"), float("inf"), float("nan")
        xs, zs = [xb.cuda()], [zb.cuda()]
        ys, ns, dx, dz = nan_like(xs), nan_like(xs, BF), nan_like(xs), nan_like(xs, BF)
        tp.tp_block_norm_fwd(xs, zs, ys, ns, **a)
        tp.tp_block_norm_bwd(zs, xs, [dn.cuda()], [dy.cuda()], dx, dz, tp.workspace(tp.TP_OP_BLOCK_NORM_BWD, 1, M, h, 0), **a)
        out.append([t[0].cpu() for t in (ys, ns, dx, dz)])
    good = [i for i in range(M) if i not in (5, 9, 20)]
    for clean, dirty in zip(*out):
        assert torch.equal(clean[good], dirty[good])
    for i in (9, 20):
        assert torch.isnan(out[1][0][i]).any() and torch.isnan(out[1][1][i]).all() and torch.isnan(out[1][3][i]).any()
    assert torch.isnan(out[1][1][5]).all() and torch.isnan(out[1][2][5]).all()


@pytest.mark.gpu
def test_constant_and_zero_rows(tp):
    """Variance zero: the deviation is sqrt(eps), and a layer norm leaves the bias."""
    M, h = 6, 520
    x, z, dn, dy, d = make(M, h, "layer", "layer", 0, F32)
    x[:], z[:] = 0, 3.0
    z[2:4] = 0
    xs, zs = [x.cuda()], [z.cuda()]
    ys, ns = nan_like(xs), nan_like(xs, BF)
    tp.tp_block_norm_fwd(xs, zs, ys, ns, **call_args(tp, d))
    y, n = ref.block_fwd(x.to(D), z.to(D), wide(d))
    close_row(cat(ys), y, torch.ones((M, 1), dtype=D), "y")
    close_row(cat(ns), n, torch.full((M, 1), 16.0, dtype=D), "n")


@pytest.mark.gpu
def test_a_mean_far_from_zero(tp):
    """A layer norm subtracts the mean before it squares: an offset of 200
    deviations costs the 8 bits by which the inputs are larger, no more."""
    M, h = 8, 2056
    g = torch.Generator().manual_seed(3)
    x = (200 + torch.randn(M, h, generator=g)).float()
    d = dict(post="none", pre="layer", w_post=None, b_post=None, w_pre=None, b_pre=None, gate=None, alpha=1.0, eps=1e-5)
    ns = [torch.empty((M, h), dtype=BF, device="cuda")]
    tp.tp_block_norm_fwd([x.cuda()], None, None, ns, **call_args(tp, d))
    n = ref.block_fwd(x.to(D), None, d)[1]
    close_row(ns[0], n, torch.full((M, 1), 210.0, dtype=D), "n")


@pytest.mark.gpu
@pytest.mark.parametrize("h", [256, 4096])
def test_in_place_on_another_stream_and_twice_the_same(tp, h):
    p, M = 2, 66
    x, z, dn, dy, d = make(M, h, "rms", "rms", 1, BF)
    a = call_args(tp, d)
    xs, zs = shards(x, p), shards(z, p)
    ys, ns = nan_like(xs), nan_like(xs, BF)
    tp.tp_block_norm_fwd(xs, zs, ys, ns, **a)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    x2, n2 = [t.clone() for t in xs], nan_like(xs, BF)
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        tp.tp_block_norm_fwd(x2, zs, x2, n2, **a)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(cat(x2), cat(ys)) and torch.equal(cat(n2), cat(ns))
    got = []
    for _ in range(2):
        dx, dz = shards(dy, p), nan_like(xs, BF)
        g = {k: torch.empty(h, device="cuda") for k in ("dw_post", "dw_pre")}
        g["dgate"] = torch.empty((1, h), device="cuda")
        tp.tp_block_norm_bwd(zs, ys, shards(dn, p), dx, dx, dz, tp.workspace(tp.TP_OP_BLOCK_NORM_BWD, p, M, h, 0), **g, **a)
        got.append([cat(dx), cat(dz), *[t.cpu() for t in g.values()]])
    assert all(torch.equal(s, t) for s, t in zip(*got))


@pytest.mark.gpu
def test_no_rows_and_graph_replay(tp):
    h = 520
    x, z, dn, dy, d = make(4, h, "layer", "rms", 1, BF)
    a = call_args(tp, d)
    e = [torch.empty((0, h), dtype=BF, device="cuda")]
    tp.tp_block_norm_fwd(e, e, e, e, **a)
    g = {k: torch.full((h,), 7.0, device="cuda") for k in ("dw_post", "db_post", "dw_pre")}
    dg = torch.full((1, h), 7.0, device="cuda")
    tp.tp_block_norm_bwd(e, e, e, e, e, e, tp.workspace(tp.TP_OP_BLOCK_NORM_BWD, 1, 0, h, 0), **g, dgate=dg, **a)
    assert all(float(t.abs().max()) == 0 for t in (*g.values(), dg))
    xs, zs = [x.cuda()], [z.cuda()]
    ys, ns = nan_like(xs), nan_like(xs, BF)
    tp.tp_block_norm_fwd(xs, zs, ys, ns, **a)
    want = [ys[0].clone(), ns[0].clone()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_block_norm_fwd(xs, zs, ys, ns, **a)
    ys[0].zero_()
    ns[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ns[0], want[1])


def test_the_formula_of_the_gradients_against_differences():
    """The 64-bit gradients that the kernels are held to, against central
    differences of the 64-bit forward pass.  With a step of 1e-5 the error of
    a difference is about 1e-10 of the third derivatives and 1e-11 of
    rounding; 1e-7 of the gradient's size is asked for."""
    M, h = 6, 24
    for post, pre, gate in (("rms", "rms", 1), ("layer", "layer", 3), ("none", "rms", 6), ("layer", "rms", 0)):
        x, z, dn, dy, d = make(M, h, post, pre, gate, F32, seed=5)
        d = wide(d)
        v = dict(x=x.to(D), z=z.to(D), **{k: d[k] for k in ("w_post", "b_post", "w_pre", "b_pre", "gate") if d[k] is not None})
        dn, dy = dn.to(D), dy.to(D)

        def loss(v):
            y, n = ref.block_fwd(v["x"], v["z"], {**d, **{k: t for k, t in v.items() if k in d}})
            return float((y * dy).sum() + (n * dn).sum())

        y = ref.block_fwd(v["x"], v["z"], d)[0]
        g = ref.block_bwd(y, v["z"], dn, dy, d)
        name = {"x": "dx", "z": "dz", "gate": "dgate"}
        for k, t in v.items():
            want = g[name.get(k, "d" + k)]
            num = torch.zeros_like(t)
            for i in range(t.numel()):
                keep = float(t.view(-1)[i])
                t.view(-1)[i] = keep + 1e-5
                up = loss(v)
                t.view(-1)[i] = keep - 1e-5
                down = loss(v)
                t.view(-1)[i] = keep
                num.view(-1)[i] = (up - down) / 2e-5
            assert float((num - want).abs().max()) <= 1e-7 * max(1.0, float(want.abs().max())), (post, pre, k)
