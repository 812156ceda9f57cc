"""What is measured of the 8-bit sharded Linear and the routed experts.

Three operators, each as a user of the library calls it and in a plain form
(elementary torch operations in 32 bits, one rounding at the end):

  route    routing of tokens to experts: softmax or sigmoid scores, a bias
           that only the choice sees, groups, top-k, renormalised weights
           (tp_route_fwd, tp_route_bwd)
  col, row, mlp
           the sharded layouts with 8-bit floating-point operands, a scale
           for each block of 128 (tp_fp8_pack, tp_{col,row}_linear_fwd_fp8,
           tp_{col,row}_linear_bwd_fp8)
  experts  the routed experts' products on the same operands, from the
           tokens' rows to their weighted sums, and the gradients
           (tp_experts_fwd_fp8, tp_experts_bwd_fp8)

Formats
  8-bit operand of a matrix [R, C] whose products sum over C: q e4m3
  [R, C rounded up to 128], zeros past C, and e uint8
  [ceil(R/128), ceil(C/512), 512], the exponents of 128 rows and four blocks
  of 128 columns: row r, block b at [r/128, b/4, r%32 * 16 + r%128/32 * 4 + b%4].
  The value is q * 2^(e - 127); 2^(e - 127) is the smallest power of two, at
  least 2^-127, whose 448-fold reaches the block's largest magnitude.  A block
  is 128 columns of a row (activations, gradients) or 128 x 128 (weights).
"""
import math

import torch

own = False

SOFTMAX, SIGMOID = "softmax", "sigmoid"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step, softmax over 64 experts: latency counts
        dict(name="route 1 token", op="route", T=1, E=64, k=6, score=SOFTMAX, bias=False, groups=1, tops=1, best=1,
             renorm=False, f32=False, train=False),
        # a training step's 8192 tokens: sigmoid scores with a balancing bias, 4 of 8 groups, top 8, and the gradient
        dict(name="route 8192 tokens groups train", op="route", T=8192, E=256, k=8, score=SIGMOID, bias=True, groups=8, tops=4,
             best=2, renorm=True, f32=False, train=True),
        # two ragged sequences, 60 experts, fp32 logits, some experts closed
        dict(name="route 1846 tokens odd train", op="route", T=1846, E=60, k=4, score=SOFTMAX, bias=False, groups=1, tops=1,
             best=1, renorm=True, f32=True, train=True),
        # single-token decode: FC1 with GeLU, the largest weights
        dict(name="col 1 token p8", op="col", p=8, M=1, N=6144, K=12288),
        # a short prompt, odd sizes: latency counts
        dict(name="row 77 tokens odd p2", op="row", p=2, M=77, N=520, K=1000),
        # 48 decode streams through the sharded MLP
        dict(name="mlp 48 tokens p4", op="mlp", p=4, M=48, h=4096, nk=4096, train=False),
        # the MLP's training step of 4096 tokens: forward and backward
        dict(name="mlp 4096 tokens p4 train", op="mlp", p=4, M=4096, h=4096, nk=4096, train=True),
        # a ragged micro-batch's training step, odd sizes
        dict(name="mlp 1100 tokens odd p2 train", op="mlp", p=2, M=1100, h=1160, nk=520, train=True),
        # one token through 6 of 64 experts: their weights' bytes
        dict(name="experts 1 token", op="experts", p=4, T=1, E=64, k=6, h=4096, f=2048, closed=False, train=False),
        # 48 decode streams: nearly every expert's weights
        dict(name="experts 48 tokens", op="experts", p=4, T=48, E=64, k=6, h=4096, f=2048, closed=False, train=False),
        # a prompt of 4096 tokens
        dict(name="experts 4096 tokens", op="experts", p=4, T=4096, E=64, k=6, h=4096, f=2048, closed=False, train=False),
        # a ragged micro-batch's training step over 16 experts, with slots left empty
        dict(name="experts 1846 tokens train", op="experts", p=2, T=1846, E=16, k=2, h=2048, f=4096, closed=True, train=True),
    ]


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], even over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v) // step * step)


def draw(rng):
    op = rng.choice(["route", "col", "row", "mlp", "experts", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 4, 256 // groups)
        tops = rng.randint(1, groups)
        score, bias = rng.choice([(SOFTMAX, False), (SIGMOID, False), (SIGMOID, True), (SOFTMAX, True)])
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E // groups * tops)), score=score, bias=bias,
                    groups=groups, tops=tops, best=rng.choice([1, 2]), renorm=rng.random() < 0.5, f32=rng.random() < 0.5,
                    train=rng.random() < 0.5)
    if op in ("col", "row"):
        while True:
            c = dict(op=op, p=rng.choice([1, 2, 4, 8]), M=_log(rng, 1, 4096), N=_log(rng, 64, 12288, 8), K=_log(rng, 64, 12288, 8))
            if c["p"] * c["N"] * c["K"] <= 8 * 6144 * 12288 and c["M"] * c["p"] * c["N"] * c["K"] <= 8 * 4096 ** 3:
                return c
    if op == "mlp":
        while True:
            c = dict(op=op, p=rng.choice([1, 2, 4, 8]), M=_log(rng, 1, 4096), h=_log(rng, 64, 8192, 8), nk=_log(rng, 64, 8192, 8),
                     train=rng.random() < 0.5)
            if c["p"] * c["h"] * c["nk"] <= 4 * 4096 ** 2 and c["M"] * c["p"] * c["h"] * c["nk"] <= 4 * 4096 ** 3:
                return c
    while True:
        p = rng.choice([1, 2, 4])
        c = dict(op=op, p=p, T=_log(rng, 1, 4096), E=p * _log(rng, 2, 64 // p), k=rng.randint(1, 6), h=_log(rng, 64, 4096, 8),
                 f=_log(rng, 64, 4096, 8), closed=rng.random() < 0.5, train=rng.random() < 0.4)
        c["k"] = min(c["k"], c["E"])
        if c["E"] * c["h"] * c["f"] <= (16 * 2048 * 4096 if c["train"] else 64 * 4096 * 2048) and \
                c["T"] * c["k"] * c["h"] * c["f"] <= (2 * 2048 if c["train"] else 6 * 4096) * 4096 * 2048:
            return c


def work(c):
    """Each input read once, each output written once, and the products' multiplications and additions."""
    op = c["op"]
    if op == "route":
        T, E, k, s = c["T"], c["E"], c["k"], 4 if c["f32"] else 2
        fwd = T * E * s + 8 * T * k + 4 * E + (4 * E if c["bias"] else 0)
        return {"bytes": fwd + (2 * T * E * s + 8 * T * k if c["train"] else 0), "flops": (20 if c["train"] else 10) * T * E}
    scaled = lambda n: n + n // 128  # noqa: E731
    if op in ("col", "row"):
        p, M, N, K = c["p"], c["M"], c["N"], c["K"]
        x, y = (M * K, p * M * N) if op == "col" else (p * M * K, M * N)
        return {"bytes": p * scaled(N * K) + 2 * x + 2 * y, "flops": 2 * p * M * N * K}
    if op == "mlp":
        p, M, h, nk = c["p"], c["M"], c["h"], c["nk"]
        w = p * h * nk
        if not c["train"]:
            return {"bytes": 2 * scaled(w) + 4 * M * h, "flops": 4 * M * w}
        # both operands of both weights, x, y, dy, dx, the weights' gradients and the pre-activations, written and read
        return {"bytes": 4 * scaled(w) + 8 * M * h + 4 * w + 4 * p * M * nk, "flops": 12 * M * w}
    T, E, k, h, f = c["T"], c["E"], c["k"], c["h"], c["f"]
    used = E * (1 - (1 - k / E) ** T)  # experts that any token goes to, were all as likely
    w = int(used * h * f)
    if not c["train"]:
        return {"bytes": 2 * scaled(w) + 4 * T * h + 8 * T * k, "flops": 4 * T * k * h * f}
    return {"bytes": 4 * scaled(w) + 8 * T * h + 4 * E * h * f + 4 * T * k * f + 14 * T * k, "flops": 12 * T * k * h * f}


# ------------------------------------------------------------------ the 8-bit format

def _pow2(e):
    """2^e as float32 for whole e in [-126, 127], by its bits; 2^-127 below."""
    return torch.where(e < -126, torch.full(e.shape, 2.0 ** -127, device=e.device), ((e.clamp(min=-126) + 127) << 23).view(torch.float32))


def _exponents(top):
    """k of the smallest power of two 2^k >= 2^-127 with top <= 448 * 2^k."""
    m, x = torch.frexp(top)
    return torch.where(m <= 0.875, x - 9, x - 8).to(torch.int32).masked_fill(top == 0, -127).clamp(min=-127)


def _quantise(v, tiles=False):
    """(q, k) of v [..., R, C] in 32 bits: q e4m3 [..., R, C'] with C' = C rounded up to 128, k int32 [..., R, C'/128]."""
    R, C = v.shape[-2:]
    v = torch.nn.functional.pad(v, (0, -C % 128))
    b = v.view(*v.shape[:-1], -1, 128)
    top = b.abs().amax(-1)
    if tiles:
        rows = torch.nn.functional.pad(top, (0, 0, 0, -R % 128))
        top = rows.view(*rows.shape[:-2], -1, 128, rows.shape[-1]).amax(-2).repeat_interleave(128, -2)[..., :R, :]
    k = _exponents(top)
    q = (b * _pow2(-k)[..., None]).to(torch.float8_e4m3fn)
    return q.view(v.shape), k


def _value(q, k):
    """The values that (q, k) stand for, in 32 bits."""
    return (q.float().view(*k.shape, 128) * _pow2(k)[..., None]).view(q.shape)


def _rounded(v, tiles=False):
    """v [..., R, C] as its 8-bit operand holds it."""
    return _value(*_quantise(v, tiles))[..., :v.shape[-1]]


def _atoms(k):
    """The exponents k [..., R, B] in the operand's order: e uint8 [..., ceil(R/128), ceil(B/4), 512]."""
    R, B = k.shape[-2:]
    e = torch.nn.functional.pad((k + 127).to(torch.uint8), (0, -B % 4, 0, -R % 128))
    e = e.view(*e.shape[:-2], e.shape[-2] // 128, 4, 32, e.shape[-1] // 4, 4)
    n = e.dim()
    e = e.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1)
    return e.reshape(*e.shape[:-3], 512).contiguous()


def _exponents_of(e, R, B):
    """k [..., R, B] of the operand's exponents."""
    v = e.view(*e.shape[:-1], 32, 4, 4)
    n = v.dim()
    v = v.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1)
    v = v.reshape(*v.shape[:-5], v.shape[-5] * 128, v.shape[-2] * 4)
    return v[..., :R, :B].to(torch.int32) - 127


def _weight(g, shape, sigma):
    """The operand of a random weight [..., R, C], with a scale for each 128 x 128."""
    q, k = _quantise(torch.randn(shape, generator=g, device="cuda") * sigma, tiles=True)
    return q, _atoms(k)


def _turned(w, R, C):
    """The operand of the transpose of an operand with a scale for each 128 x 128: the same values."""
    v = _value(w[0], _exponents_of(w[1], R, -(-C // 128)))[..., :C].transpose(-1, -2).contiguous()
    k = _exponents_of(w[1], R, -(-C // 128))[..., ::128, :].transpose(-1, -2).repeat_interleave(128, -2)[..., :C, :]
    v = torch.nn.functional.pad(v, (0, -R % 128))
    q = (v.view(*k.shape, 128) * _pow2(-k)[..., None]).to(torch.float8_e4m3fn)
    return q.view(v.shape), _atoms(k.contiguous())


def _matrix(w, cols):
    """The values of an operand, in 32 bits, without the columns past `cols`."""
    q, e = w
    return _value(q, _exponents_of(e, q.shape[-2], q.shape[-1] // 128))[..., :cols]


# ------------------------------------------------------------------ inputs

def _normal(g, shape, sigma=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _activation(g, shape):
    """Normal values with a few columns ten times as large, as hidden states have."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[:, torch.rand(shape[1], generator=g, device="cuda") < 0.01] *= 10
    return x.to(torch.bfloat16)


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    buf = lambda shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "route":
        T, E, k = c["T"], c["E"], c["k"]
        dtype = torch.float32 if c["f32"] else torch.bfloat16
        s["logits"] = _normal(g, (T, E), 1.5, dtype)
        if c["f32"]:  # closed experts, and a row that leaves nothing
            s["logits"][torch.rand((T, E), generator=g, device="cuda") < 0.02] = -math.inf
            if T > 4:
                s["logits"][T // 2] = -math.inf
        s["bias"] = _normal(g, (E,), 0.1, torch.float32) if c["bias"] else None
        s["dweights"] = _normal(g, (T, k), 1.0, torch.float32)
        s["experts"], s["weights"] = buf((T, k), torch.int32), buf((T, k), torch.float32)
        s["counts"], s["dlogits"] = buf((E,), torch.int32), buf((T, E), dtype)
        return s
    p = c["p"]
    if op in ("col", "row"):
        M, N, K = c["M"], c["N"], c["K"]
        s["x"] = [_activation(g, (M, K)) for _ in range(p if op == "row" else 1)]
        s["w"] = [_weight(g, (N, K), 0.02) for _ in range(p)]
        s["y"] = [buf((M, N)) for _ in range(1 if op == "row" else p)]
        return s
    if op == "mlp":
        M, h, nk = c["M"], c["h"], c["nk"]
        s["x"] = _activation(g, (M, h))
        s["w1"] = [_weight(g, (nk, h), 0.02) for _ in range(p)]
        s["w2"] = [_weight(g, (h, nk), 0.02) for _ in range(p)]
        s["y"] = buf((M, h))
        if c["train"]:
            s["dy"] = _normal(g, (M, h))
            s["w1t"] = [_turned(w, nk, h) for w in s["w1"]]
            s["w2t"] = [_turned(w, h, nk) for w in s["w2"]]
            s["preact"], s["dh"] = [buf((M, nk)) for _ in range(p)], [buf((M, nk)) for _ in range(p)]
            s["dx"] = buf((M, h))
            s["dw1"], s["dw2"] = [buf((h, nk)) for _ in range(p)], [buf((nk, h)) for _ in range(p)]
        return s
    T, E, k, h, f = c["T"], c["E"], c["k"], c["h"], c["f"]
    s["x"] = _activation(g, (T, h))
    popular = torch.randn(E, generator=g, device="cuda") * 0.3
    score = torch.randn((T, E), generator=g, device="cuda") + popular
    top = torch.sort(score, dim=1, descending=True, stable=True)
    s["experts"] = top.indices[:, :k].to(torch.int32).contiguous()
    s["weights"] = torch.softmax(top.values[:, :k], 1).contiguous()
    if c["closed"]:
        none = torch.rand((T, k), generator=g, device="cuda") < 0.03
        s["experts"][none], s["weights"][none] = -1, 0.0
    # the most rows of an expert, at least one: the plain form's products are as tall for each of them
    s["most"] = max(1, int(torch.bincount(s["experts"].flatten().long() + 1, minlength=E + 1)[1:].max()))
    s["w1"] = [_weight(g, (E // p, f, h), 0.02) for _ in range(p)]
    s["w2"] = [_weight(g, (E // p, h, f), 0.02) for _ in range(p)]
    s["y"] = buf((T, h))
    if c["train"]:
        s["dy"] = _normal(g, (T, h))
        s["w1t"] = [_turned(w, f, h) for w in s["w1"]]
        s["w2t"] = [_turned(w, h, f) for w in s["w2"]]
        s["dx"], s["dweights"] = buf((T, h)), buf((T, k))
        s["dw1"], s["dw2"] = [buf((E // p, h, f)) for _ in range(p)], [buf((E // p, f, h)) for _ in range(p)]
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gemm_reduce_fusion_gb300 as tp
    c, op = s["case"], s["case"]["op"]
    if op == "route":
        how = dict(score=tp.TP_ROUTE_SIGMOID if c["score"] == SIGMOID else tp.TP_ROUTE_SOFTMAX, renorm=c["renorm"], scale=2.5)
        tp.tp_route_fwd(s["logits"], s["experts"], s["weights"], counts=s["counts"], bias=s["bias"], groups=c["groups"],
                        top_groups=c["tops"], group_best=c["best"], **how)
        if not c["train"]:
            return s["experts"], s["weights"], s["counts"]
        tp.tp_route_bwd(s["logits"], s["experts"], s["dweights"], s["dlogits"], **how)
        return s["experts"], s["weights"], s["counts"], s["dlogits"]
    p = c["p"]
    fp8 = lambda ts: [tp.Fp8(*t) for t in ts]  # noqa: E731
    if op in ("col", "row"):
        M, N, K = c["M"], c["N"], c["K"]
        if "ws" not in s:
            s["ws"] = tp.workspace(tp.TP_OP_COL_FP8 if op == "col" else tp.TP_OP_ROW_FP8, p, M, N, K)
            s["xq"] = [tp.fp8_empty(M, K) for _ in s["x"]]
        tp.tp_fp8_pack(s["x"], s["xq"])
        if op == "col":
            tp.tp_col_linear_fwd_fp8(s["xq"][0], fp8(s["w"]), s["y"], s["ws"], epi=tp.TP_EPI_GELU)
        else:
            tp.tp_row_linear_fwd_fp8(s["xq"], fp8(s["w"]), s["y"][0], s["ws"])
        return s["y"]
    if op == "mlp":
        M, h, nk, train = c["M"], c["h"], c["nk"], c["train"]
        if "ws" not in s:
            ops = [(tp.TP_OP_COL_FP8, p, M, nk, h), (tp.TP_OP_ROW_FP8, p, M, h, nk)]
            if train:
                ops += [(tp.TP_OP_ROW_BWD_FP8, p, M, h, nk), (tp.TP_OP_COL_BWD_FP8, p, M, nk, h)]
            s["ws"] = max((tp.workspace(*o) for o in ops), key=lambda w: w.numel())
            s["xq"], s["zq"] = tp.fp8_empty(M, h), [tp.fp8_empty(M, nk) for _ in range(p)]
            if train:
                s["xt"], s["zt"] = tp.fp8_empty(h, M), [tp.fp8_empty(nk, M) for _ in range(p)]
                s["dyq"], s["dyt"] = tp.fp8_empty(M, h), tp.fp8_empty(h, M)
                s["dhq"], s["dht"] = [tp.fp8_empty(M, nk) for _ in range(p)], [tp.fp8_empty(nk, M) for _ in range(p)]
        tp.tp_fp8_pack([s["x"]], [s["xq"]], [s["xt"]] if train else None)
        tp.tp_col_linear_fwd_fp8(s["xq"], fp8(s["w1"]), None, s["ws"], epi=tp.TP_EPI_GELU, z=s["zq"],
                                 preact=s["preact"] if train else None)
        tp.tp_row_linear_fwd_fp8(s["zq"], fp8(s["w2"]), s["y"], s["ws"])
        if not train:
            return s["y"]
        tp.tp_fp8_pack([s["dy"]], [s["dyq"]], [s["dyt"]])
        tp.tp_fp8_pack(s["preact"], None, s["zt"], epi=tp.TP_EPI_GELU)
        tp.tp_row_linear_bwd_fp8(s["zt"], fp8(s["w2t"]), s["dyq"], s["dyt"], s["dh"], s["dw2"], s["ws"], preact=s["preact"])
        tp.tp_fp8_pack(s["dh"], s["dhq"], s["dht"])
        tp.tp_col_linear_bwd_fp8(s["xt"], fp8(s["w1t"]), s["dhq"], s["dht"], s["dx"], s["dw1"], s["ws"])
        return s["y"], s["preact"], s["dx"], s["dw1"], s["dw2"]
    T, E, k, h, f = c["T"], c["E"], c["k"], c["h"], c["f"]
    if "ws" not in s:
        s["ws"] = tp.experts_workspace(p, E, T, k, h, f, backward=c["train"])
        s["saved"] = tp.experts_saved(E, T, k, h, f) if c["train"] else None
    tp.tp_experts_fwd_fp8(s["x"], s["experts"], s["weights"], fp8(s["w1"]), fp8(s["w2"]), s["y"], s["ws"], saved=s["saved"])
    if not c["train"]:
        return s["y"]
    tp.tp_experts_bwd_fp8(s["x"], s["weights"], s["dy"], fp8(s["w1t"]), fp8(s["w2t"]), s["dx"], s["dweights"], s["dw1"], s["dw2"],
                          s["saved"], s["ws"])
    return s["y"], s["dx"], s["dweights"], s["dw1"], s["dw2"]


def _gelu(x):
    return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))


def _gelu_prime(x):
    return 0.5 * (1 + torch.erf(x * 0.5 ** 0.5)) + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))


def _scores(s):
    """(open, scores) in 64 bits, where the choice between near ones is made: an expert with a logit of -inf is closed."""
    l = s["logits"].double()
    open_ = l > -math.inf
    l = l.masked_fill(~open_, -math.inf)
    if s["case"]["score"] == SIGMOID:
        return open_, 1 / (1 + torch.exp(-l))
    top = l.amax(1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(l - top)
    return open_, e / e.sum(1, keepdim=True).clamp(min=1e-38)


def _route_plain(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    open_, sc = _scores(s)
    v = sc if s["bias"] is None else sc + s["bias"].double()
    v = v.masked_fill(~open_, -math.inf)
    if c["groups"] > 1:
        best = v.view(T, c["groups"], -1).sort(2, descending=True).values[..., :c["best"]]
        any_ = best[..., 0] > -math.inf
        best = best.masked_fill(best == -math.inf, 0).sum(2).masked_fill(~any_, -math.inf)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["tops"]]
        keep = torch.zeros_like(any_).scatter(1, kept, True)
        v = v.masked_fill(~keep.repeat_interleave(E // c["groups"], 1), -math.inf)
    top = torch.sort(v, dim=1, descending=True, stable=True)
    at, there = top.indices[:, :k], top.values[:, :k] > -math.inf
    w = sc.gather(1, at) * there
    total = w.sum(1, keepdim=True).clamp(min=1e-38) if c["renorm"] else torch.ones((T, 1), dtype=w.dtype, device=w.device)
    experts = at.masked_fill(~there, -1)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=w.device).index_add(
        0, (experts + 1).flatten(), torch.ones(T * k, dtype=torch.int32, device=w.device))[1:]
    out = experts.to(torch.int32), (2.5 * w / total).float(), counts
    if not c["train"]:
        return out
    g = 2.5 * s["dweights"].double() * there
    if c["renorm"]:
        g = (g - (g * w).sum(1, keepdim=True) / total) / total * there
    ds = torch.zeros_like(sc).scatter_add(1, at, g)
    d = ds * sc * (1 - sc) if c["score"] == SIGMOID else sc * (ds - (ds * sc).sum(1, keepdim=True))
    return (*out, d.to(s["logits"].dtype))


def _rows_of(s):
    """The rows that the slots (token, choice) take among their experts' rows, in the order of tokens: (row, there), both [T * k]."""
    c = s["case"]
    e = s["experts"].flatten().long()
    hot = torch.zeros((e.numel(), c["E"] + 1), dtype=torch.int32, device=e.device).scatter_(1, (e + 1)[:, None], 1)
    rank = (hot.cumsum(0) - 1).gather(1, (e + 1)[:, None])[:, 0]
    return e.clamp(min=0) * s["most"] + rank.clamp(max=s["most"] - 1), e >= 0


def _spread(v, row, there, n):
    """v [slots, C] at its rows of n, zeros elsewhere."""
    out = torch.zeros((n + 1, v.shape[1]), dtype=v.dtype, device=v.device)
    return out.index_copy(0, torch.where(there, row, torch.full_like(row, n)), v)[:n] if n else out[:0]


def _run_plain(s):
    c, op, bf = s["case"], s["case"]["op"], torch.bfloat16
    if op == "route":
        return _route_plain(s)
    p = c["p"]
    if op in ("col", "row"):
        w = [_matrix(a, c["K"]) for a in s["w"]]
        x = [_rounded(a.float()) for a in s["x"]]
        if op == "row":
            return [(torch.cat(x, 1) @ torch.cat(w, 1).t()).to(bf)]
        return [_gelu(x[0] @ a.t()).to(bf) for a in w]
    if op == "mlp":
        M, h, nk = c["M"], c["h"], c["nk"]
        w1, w2 = torch.stack([_matrix(a, h) for a in s["w1"]]), torch.stack([_matrix(a, nk) for a in s["w2"]])
        hh = _rounded(s["x"].float()) @ w1.transpose(1, 2)
        z = _rounded(_gelu(hh))
        y = (z.transpose(0, 1).reshape(M, -1) @ w2.transpose(0, 1).reshape(h, -1).t()).to(bf)
        if not c["train"]:
            return y
        hh = hh.to(bf)  # as it is saved
        zt = _rounded(_gelu(hh.float()).transpose(1, 2))
        dyq, dyt, xt = _rounded(s["dy"].float()), _rounded(s["dy"].float().t()), _rounded(s["x"].float().t())
        dh = ((dyq @ w2) * _gelu_prime(hh.float())).to(bf)
        dw2 = zt @ dyt.t()
        dx = _rounded(dh.float()).transpose(0, 1).reshape(M, -1) @ w1.reshape(-1, h)
        dw1 = xt @ _rounded(dh.float().transpose(1, 2)).transpose(1, 2)
        return y, list(hh), dx.to(bf), list(dw1.to(bf)), list(dw2.to(bf))
    T, E, k, h, f, most = c["T"], c["E"], c["k"], c["h"], c["f"], s["most"]
    w1, w2 = torch.cat([_matrix(a, h) for a in s["w1"]]), torch.cat([_matrix(a, f) for a in s["w2"]])
    row, there = _rows_of(s)
    x = s["x"].float()
    xs = _spread(x.repeat_interleave(k, 0), row, there, E * most).view(E, most, h)
    hh = _rounded(xs) @ w1.transpose(1, 2)
    o = _rounded(_gelu(hh)) @ w2.transpose(1, 2)
    mine = o.view(-1, h)[row].view(T, k, h)
    wt = (s["weights"].flatten() * there).view(T, k)
    y = (mine * wt[..., None]).sum(1).to(bf)
    if not c["train"]:
        return y
    hh = hh.to(bf).float()  # as it is saved
    dy = s["dy"].float()
    dw = ((mine.to(bf).float() * dy[:, None]).sum(2) * there.view(T, k)).to(bf)
    do = _spread((wt[..., None] * dy[:, None]).view(-1, h), row, there, E * most).view(E, most, h)
    dh = ((_rounded(do) @ w2) * _gelu_prime(hh)).to(bf).float()
    dxs = _rounded(dh) @ w1
    dx = (dxs.view(-1, h)[row] * there[:, None]).view(T, k, h).sum(1).to(bf)
    dw2 = _rounded(_gelu(hh).transpose(1, 2)) @ _rounded(do.transpose(1, 2)).transpose(1, 2)
    dw1 = _rounded(xs.transpose(1, 2)) @ _rounded(dh.transpose(1, 2)).transpose(1, 2)
    return y, dx, dw, list(dw1.to(bf).chunk(p)), list(dw2.to(bf).chunk(p))


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    """What run returns for these inputs, from the definitions, in 64 bits."""
    c, s = case, prepare(case, seed)
    D, bf = torch.float64, torch.bfloat16

    def two_to(e):  # by its bits
        return ((e.to(torch.int64) + 1023) << 52).view(D)

    def held(v):
        """v [R, C] as e4m3 values with a power of two for every 128 columns of a row, by arithmetic on the grid."""
        R, C = v.shape
        u = torch.zeros((R, -(-C // 128) * 128), dtype=D, device=v.device)
        u[:, :C] = v.to(D)
        u = u.view(R, -1, 128)
        top = u.abs().amax(2)
        k = torch.ceil(torch.log2(top / 448)).clamp(min=-127)
        k = torch.where(top > 448 * two_to(k), k + 1, k)
        k = torch.where((top <= 448 * two_to(k - 1)) & (k > -127), k - 1, k)
        t = u / two_to(k)[..., None]
        x = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)))
        x = torch.where(t.abs() >= two_to(x + 1), x + 1, torch.where(t.abs() < two_to(x), x - 1, x)).clamp(min=-6)
        step = two_to(x - 3)
        return (torch.round(t / step) * step * two_to(k)[..., None]).view(R, -1)[:, :C]

    def stands_for(q, e, cols):
        """The values of an operand [R, C'], element by element from its description."""
        r = torch.arange(q.shape[0], device=q.device)[:, None]
        b = torch.arange(q.shape[1] // 128, device=q.device)[None, :]
        k = e[r // 128, b // 4, r % 32 * 16 + r % 128 // 32 * 4 + b % 4].to(torch.int64) - 127
        return (q.to(D).view(q.shape[0], -1, 128) * two_to(k)[..., None]).view(q.shape)[:, :cols]

    def phi(v):
        return torch.special.erfc(-v / math.sqrt(2)) / 2

    def slope(v):
        return phi(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)

    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        l = s["logits"].to(D)
        shut = torch.isneginf(l)
        if c["score"] == SIGMOID:
            sc = torch.special.expit(l)
        else:
            sc = torch.exp(l - torch.logsumexp(l, 1, keepdim=True)).nan_to_num(0.0)
        v = torch.where(shut, torch.full_like(l, -math.inf), sc if s["bias"] is None else sc + s["bias"].to(D))
        G, size = c["groups"], E // c["groups"]

        def first_largest(m, n):
            """The columns of the n largest, one by one; the first of equal ones; E or G past what is there."""
            m, out = m.clone(), []
            for _ in range(n):
                top = m.amax(1, keepdim=True)
                at = (m == top).to(torch.int8).argmax(1, keepdim=True)
                out.append(torch.where(top == -math.inf, torch.full_like(at, -1), at))
                m.scatter_(1, at, -math.inf)
            return torch.cat(out, 1)

        if G > 1:
            score = torch.full((T, G), -math.inf, dtype=D, device=l.device)
            for g in range(G):
                part = v[:, g * size:(g + 1) * size].clone()
                for i in range(min(c["best"], size)):
                    top, at = part.max(1)
                    score[:, g] = torch.where(top == -math.inf, score[:, g], top if i == 0 else score[:, g] + top)
                    part.scatter_(1, at[:, None], -math.inf)
            chosen = first_largest(score, c["tops"])
            group = torch.arange(E, device=l.device) // size
            v = torch.where((group[None, :, None] == chosen[:, None, :]).any(2), v, torch.full_like(v, -math.inf))
        experts = first_largest(v, k)
        w = torch.where(experts < 0, torch.zeros((), dtype=D, device=l.device), sc.gather(1, experts.clamp(min=0)))
        n = w.sum(1, keepdim=True) if c["renorm"] else torch.ones((T, 1), dtype=D, device=l.device)
        n = torch.where(n == 0, torch.ones_like(n), n)
        counts = (experts[:, :, None] == torch.arange(E, device=l.device)).sum((0, 1)).to(torch.int32)
        out = experts.to(torch.int32), 2.5 * w / n, counts
        if not c["train"]:
            return out
        g = torch.where(experts < 0, torch.zeros((), dtype=D, device=l.device), s["dweights"].to(D)) * 2.5
        if c["renorm"]:
            g = g / n - (g * w).sum(1, keepdim=True) / n ** 2
        d = torch.zeros_like(sc)
        for i in range(k):
            at = experts[:, i:i + 1]
            d.scatter_add_(1, at.clamp(min=0), torch.where(at < 0, torch.zeros_like(g[:, i:i + 1]), g[:, i:i + 1]))
        d = d * sc * (1 - sc) if c["score"] == SIGMOID else sc * d - sc * (sc * d).sum(1, keepdim=True)
        return (*out, d)
    p = c["p"]
    if c["op"] in ("col", "row"):
        w = [stands_for(q, e, c["K"]) for q, e in s["w"]]
        x = [held(a) for a in s["x"]]
        if c["op"] == "row":
            return [sum(a @ b.t() for a, b in zip(x, w))]
        return [(x[0] @ b.t()) * phi(x[0] @ b.t()) for b in w]
    if c["op"] == "mlp":
        h, nk = c["h"], c["nk"]
        x, y, saved, dx, dw1, dw2 = held(s["x"]), 0, [], 0, [], []
        for k in range(p):
            w1, w2 = stands_for(*s["w1"][k], h), stands_for(*s["w2"][k], nk)
            a = x @ w1.t()
            y = y + held(a * phi(a)) @ w2.t()
            if c["train"]:
                a = a.to(bf).to(D)
                saved.append(a)
                dh = ((held(s["dy"]) @ w2) * slope(a)).to(bf).to(D)
                dx = dx + held(dh) @ w1
                dw1.append(held(s["x"].t()) @ held(dh.t()).t())
                dw2.append(held((a * phi(a)).t()) @ held(s["dy"].t()).t())
        return (y, saved, dx, dw1, dw2) if c["train"] else y
    T, E, k, h, f = c["T"], c["E"], c["k"], c["h"], c["f"]
    x, dy = s["x"].to(D), s["dy"].to(D) if c["train"] else None
    y, dx = torch.zeros((T, h), dtype=D, device="cuda"), torch.zeros((T, h), dtype=D, device="cuda")
    dw = torch.zeros((T, k), dtype=D, device="cuda")
    dw1 = torch.zeros((E, h, f), dtype=D, device="cuda") if c["train"] else None
    dw2 = torch.zeros((E, f, h), dtype=D, device="cuda") if c["train"] else None
    for e in range(E):
        t, j = (s["experts"] == e).nonzero(as_tuple=True)  # in the order of tokens
        if not t.numel():
            continue
        w1 = stands_for(s["w1"][e // (E // p)][0][e % (E // p)], s["w1"][e // (E // p)][1][e % (E // p)], h)
        w2 = stands_for(s["w2"][e // (E // p)][0][e % (E // p)], s["w2"][e // (E // p)][1][e % (E // p)], f)
        a = held(x[t]) @ w1.t()
        o = held(a * phi(a)) @ w2.t()
        wt = s["weights"][t, j][:, None]
        y.index_add_(0, t, wt.to(D) * o)
        if c["train"]:
            a = a.to(bf).to(D)
            dw[t, j] = (o.to(bf).to(D) * dy[t]).sum(1)
            do = (wt * s["dy"][t].float()).to(D)  # rounded to 32 bits, as it is before it is held in 8
            dh = ((held(do) @ w2) * slope(a)).to(bf).to(D)
            dx.index_add_(0, t, held(dh) @ w1)
            dw1[e] = held(x[t].t()) @ held(dh.t()).t()
            dw2[e] = held((a * phi(a)).t()) @ held(do.t()).t()
    return (y, dx, dw, list(dw1.chunk(p)), list(dw2.chunk(p))) if c["train"] else y
