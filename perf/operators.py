"""What is measured of the operators around the sharded Linear.

Four operators of a tensor-parallel transformer block, each as a user of the
library calls it and in a plain form (elementary torch operations in 32 bits,
one rounding at the end):

  norm_fwd     y = x + alpha * gate * N_post(z), n = N_pre(y): the boundary
               between two blocks (tp_block_norm_fwd)
  norm_bwd     its gradients (tp_block_norm_bwd)
  ckpt         activations saved in 8 bits in the forward pass and restored in
               the backward pass, optionally through GeLU (tp_ckpt_pack,
               tp_ckpt_unpack)
  row_bwd_ckpt, col_bwd_ckpt
               the backward passes of the two sharded layouts on such
               checkpoints (tp_row_linear_bwd_ckpt, tp_col_linear_bwd_ckpt)
  col_w4, row_w4
               both forward layouts for a few tokens with 4-bit weights
               (tp_col_linear_fwd_w4, tp_row_linear_fwd_w4)

Formats
  checkpoint   q int8 [M, N] and e uint8 [M, ceil(N/32)]: the value is
               q * 2^(e - 126) for each group of 32 columns; e = 255 marks a
               group that held an infinity or NaN and stands for NaN
  4-bit        q uint8 [ceil(N/32), ceil(K/64), 1024] and s bf16
               [ceil(N/32), ceil(K/G), 32]; see _w4_plain for the order
"""
import math

import torch

own = False

RMS, LAYER = "rms", "layer"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step through the boundary of two blocks: latency counts
        dict(name="norm_fwd 1 token", op="norm_fwd", p=1, M=1, h=4096, post=RMS, pre=RMS, gate=1, res32=False),
        # 8192 tokens, sequence-parallel over 8 ranks: the training and prompt shape
        dict(name="norm_fwd 8192x8192 p8", op="norm_fwd", p=8, M=8192, h=8192, post=RMS, pre=RMS, gate=1, res32=False),
        # two ragged sequences, each with a gate of its own, layer norms with biases, an fp32 residual stream
        dict(name="norm_bwd 1846x1160 odd", op="norm_bwd", p=1, M=1846, h=1160, post=LAYER, pre=LAYER, gate=2, res32=True),
        # the largest hidden size, 2048 tokens over 8 ranks: the backward pass of a training step
        dict(name="norm_bwd 2048x12288 p8", op="norm_bwd", p=8, M=2048, h=12288, post=RMS, pre=RMS, gate=1, res32=False),
        # a short micro-batch with odd sizes: saved, then restored as it was
        dict(name="ckpt 333x1000 p2", op="ckpt", p=2, M=333, N=1000, gelu=False),
        # the MLP's pre-activations of 4096 tokens, 4 shards: saved, then restored through GeLU
        dict(name="ckpt 4096x4096 p4 gelu", op="ckpt", p=4, M=4096, N=4096, gelu=True),
        # FC2's backward pass from saved pre-activations, the MLP training shape
        dict(name="row_bwd_ckpt mlp p4", op="row_bwd_ckpt", p=4, M=4096, N=4096, K=4096),
        # a column layer's backward pass from its saved input, odd sizes
        dict(name="col_bwd_ckpt odd p2", op="col_bwd_ckpt", p=2, M=1100, N=520, K=1160),
        # single-token decode: FC1 with GeLU, the largest weights
        dict(name="col_w4 1 token p8", op="col_w4", p=8, M=1, N=6144, K=12288, G=128, gelu=True, f32=False),
        # 16 decode streams: FC2 with its reduction over the ranks
        dict(name="row_w4 16 tokens p8", op="row_w4", p=8, M=16, N=12288, K=6144, G=64, gelu=False, f32=False),
        # 5 streams, odd sizes, small groups, fp32 output: latency counts
        dict(name="row_w4 5 tokens odd p2", op="row_w4", p=2, M=5, N=520, K=1000, G=32, gelu=False, f32=True),
        # 48 streams on the MLP training shape's FC1
        dict(name="col_w4 48 tokens p4", op="col_w4", p=4, M=48, N=4096, K=4096, G=128, gelu=True, f32=False),
    ]


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], even over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v) // step * step)


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "ckpt", "row_bwd_ckpt", "col_bwd_ckpt", "col_w4", "row_w4"])
    p = rng.choice([1, 2, 4, 8])
    if op in ("norm_fwd", "norm_bwd"):
        h = _log(rng, 64, 12288, 8)
        most = 8192 * 8192 if op == "norm_fwd" else 2048 * 12288
        mp = _log(rng, 1, max(1, min(8192, most // h) // p))
        M = mp * p
        gate = rng.choice([0, 1, p, M])
        return dict(op=op, p=p, M=M, h=h, post=rng.choice([RMS, LAYER, "none"]), pre=rng.choice([RMS, LAYER]), gate=gate,
                    res32=rng.random() < 0.3)
    if op == "ckpt":
        N = _log(rng, 64, 12288, 8)
        return dict(op=op, p=p, M=_log(rng, 1, max(1, min(8192, 4 * 4096 * 4096 // (N * p)))), N=N, gelu=rng.random() < 0.5)
    if op in ("row_bwd_ckpt", "col_bwd_ckpt"):
        while True:
            c = dict(op=op, p=p, M=_log(rng, 16, 4096), N=_log(rng, 64, 4096, 8), K=_log(rng, 64, 4096, 8))
            if c["p"] * c["M"] * c["N"] * c["K"] <= 4 * 4096 ** 3:
                return c
    while True:
        c = dict(op=op, p=p, M=_log(rng, 1, 64), N=_log(rng, 128, 12288, 8), K=_log(rng, 128, 12288, 8),
                 G=rng.choice([32, 64, 128]), gelu=op == "col_w4" and rng.random() < 0.5, f32=rng.random() < 0.3)
        if c["p"] * c["N"] * c["K"] <= 8 * 6144 * 12288 and c["M"] * c["p"] * c["N"] * c["K"] <= 16 * 8 * 6144 * 12288:
            return c


def work(c):
    """Each input read once, each output written once, and the products' multiplications and additions."""
    op, p = c["op"], c["p"]
    if op in ("norm_fwd", "norm_bwd"):
        M, h, r = c["M"], c["h"], 4 if c["res32"] else 2
        vectors = h * ((2 if c["post"] == LAYER else 1 if c["post"] == RMS else 0) + (2 if c["pre"] == LAYER else 1))
        gate = c["gate"] * h
        if op == "norm_fwd":
            return {"bytes": M * h * (2 * r + 4) + 2 * (vectors + gate), "flops": 12 * M * h}
        return {"bytes": M * h * (3 * r + 6) + 6 * (vectors + gate), "flops": 30 * M * h}
    if op == "ckpt":
        M, N = c["M"], c["N"]
        return {"bytes": p * M * (2 * N + 2 * N + 2 * (N + -(-N // 32))), "flops": 4 * p * M * N}
    M, N, K = c["M"], c["N"], c["K"]
    if op == "row_bwd_ckpt":
        return {"bytes": p * M * (K + -(-K // 32)) + 2 * (p * K * N * 2 + M * N + p * M * K), "flops": 4 * p * M * N * K}
    if op == "col_bwd_ckpt":
        return {"bytes": M * (K + -(-K // 32)) + 2 * (p * K * N * 2 + p * M * N + M * K), "flops": 4 * p * M * N * K}
    size = 4 if c["f32"] else 2
    x, y = (M * K, p * M * N) if op == "col_w4" else (p * M * K, M * N)
    return {"bytes": p * (K * N // 2 + 2 * N * -(-K // c["G"])) + 2 * x + size * y, "flops": 2 * p * M * N * K}


# ------------------------------------------------------------------ inputs

def _normal(g, shape, sigma=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _activation(g, shape):
    """Normal values with a few columns ten times as large, as hidden states have."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[:, torch.rand(shape[1], generator=g, device="cuda") < 0.01] *= 10
    return x.to(torch.bfloat16)


def _pow2(e):
    """2^e as float32 for whole e in [-126, 127], by its bits."""
    return ((e + 127) << 23).view(torch.float32)


def _pack_plain(x):
    """q int8 and e uint8 of x [M, N]: the smallest power of two whose 127-fold reaches the group's largest value."""
    M, N = x.shape
    g = -(-N // 32)
    v = torch.zeros((M, g * 32), device=x.device)
    v[:, :N] = x
    v = v.view(M, g, 32)
    top = v.abs().amax(2)
    bad = ~torch.isfinite(v).all(2)
    top = torch.where(bad, torch.zeros_like(top), top)
    m, k = torch.frexp(top)
    e = torch.where(m <= 127 / 128, k - 7, k - 6).to(torch.int32).clamp(min=-126)
    q = torch.round(v * _pow2(-e)[..., None])
    q = torch.where(bad[..., None], torch.zeros_like(q), q).to(torch.int8)
    return q.view(M, g * 32)[:, :N].contiguous(), torch.where(bad, torch.full_like(e, 255), e + 126).to(torch.uint8)


def _unpack_plain(q, e):
    M, N = q.shape
    s = torch.where(e == 255, torch.full(e.shape, float("nan"), device=q.device), _pow2(e.to(torch.int32).clamp(max=253) - 126))
    return q.float() * s.repeat_interleave(32, 1)[:, :N]


def prepare(case, seed):
    c, p = case, case["p"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    bf, f32 = torch.bfloat16, torch.float32
    buf = lambda shape, dtype=bf: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] in ("norm_fwd", "norm_bwd"):
        M, h, res = c["M"], c["h"], f32 if c["res32"] else bf
        m = M // p
        near_one = lambda: (1 + 0.1 * torch.randn(h, generator=g, device="cuda")).to(bf)  # noqa: E731
        s["alpha"] = 0.5
        s["z"] = [_activation(g, (m, h)) for _ in range(p)]
        s["w_post"] = near_one() if c["post"] != "none" else None
        s["b_post"] = _normal(g, (h,), 0.1) if c["post"] == LAYER else None
        s["w_pre"] = near_one()
        s["b_pre"] = _normal(g, (h,), 0.1) if c["pre"] == LAYER else None
        s["gate"] = _normal(g, (c["gate"], h), 0.5) if c["gate"] else None
        stream = [(_activation(g, (m, h)).float() * 2).to(res) for _ in range(p)]
        if c["op"] == "norm_fwd":
            s["x"] = stream
            s["y"] = [buf((m, h), res) for _ in range(p)]
            s["n"] = [buf((m, h)) for _ in range(p)]
        else:
            s["y"] = stream
            s["dn"] = [_normal(g, (m, h)) for _ in range(p)]
            s["dy"] = [_normal(g, (m, h), 1.0, res) for _ in range(p)]
            s["dx"] = [buf((m, h), res) for _ in range(p)]
            s["dz"] = [buf((m, h)) for _ in range(p)]
            for k, like in (("dw_post", "w_post"), ("db_post", "b_post"), ("dw_pre", "w_pre"), ("db_pre", "b_pre"), ("dgate", "gate")):
                s[k] = buf(s[like].shape, f32) if s[like] is not None else None
            s["ws"] = _workspace("BLOCK_NORM_BWD", p, M, h, 0)
        return s
    if c["op"] == "ckpt":
        M, N = c["M"], c["N"]
        s["x"] = [_activation(g, (M, N)) for _ in range(p)]
        s["q"] = [buf((M, N), torch.int8) for _ in range(p)]
        s["e"] = [buf((M, -(-N // 32)), torch.uint8) for _ in range(p)]
        s["y"] = [buf((M, N)) for _ in range(p)]
        return s
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] in ("row_bwd_ckpt", "col_bwd_ckpt"):
        row = c["op"] == "row_bwd_ckpt"
        saved = [_pack_plain(_activation(g, (M, K))) for _ in range(p if row else 1)]
        s["q"], s["e"] = [a for a, _ in saved], [b for _, b in saved]
        s["w"] = [_normal(g, (K, N), 0.02) for _ in range(p)]
        s["dy"] = [_normal(g, (M, N)) for _ in range(1 if row else p)]
        s["dx"] = [buf((M, K)) for _ in range(p if row else 1)]
        s["dw"] = [buf((K, N)) for _ in range(p)]
        s["ws"] = _workspace("ROW_BWD_CKPT" if row else "COL_BWD_CKPT", p, M, N, K)
        return s
    row, G = c["op"] == "row_w4", c["G"]
    s["x"] = [_activation(g, (M, K)) for _ in range(p if row else 1)]
    s["q"], s["s"] = [], []
    for _ in range(p):  # nibbles as rounding normal weights gives them: 8 stands for zero, and past the weights' edges all are 8
        tall, wide = -(-K // 64) * 64, -(-N // 32) * 32
        n = (torch.randn((tall, wide), generator=g, device="cuda", dtype=bf) * 2.7 + 8).round().clamp(1, 15).to(torch.int32)
        n[K:], n[:, N:] = 8, 8
        # k = 64 b + 32 d + 8 t + 4 j + 2 u + v,  n = 32 a + 16 f + 8 r + i
        n = n.view(tall // 64, 2, 4, 2, 2, 2, wide // 32, 2, 2, 8)
        n = n.permute(6, 0, 7, 9, 2, 1, 3, 5, 4, 8).reshape(wide // 32, tall // 64, 256, 8)  # [a, b, (f, i, t, d, j), (v, u, r)]
        word = torch.zeros(n.shape[:3], dtype=torch.int32, device="cuda")
        for k in range(8):
            word |= n[..., k] << (4 * k)
        s["q"].append(word.view(torch.uint8).view(wide // 32, tall // 64, 1024))
        s["s"].append((0.02 / 2.7 * torch.exp(0.2 * torch.randn((wide // 32, -(-K // G), 32), generator=g, device="cuda"))).to(bf))
    out = torch.float32 if c["f32"] else bf
    s["out"] = [buf((M, N), out) for _ in range(1 if row else p)]
    s["ws"] = _workspace("ROW_W4" if row else "COL_W4", p, M, N, K)
    return s


def _workspace(op, *sizes):
    """The library's workspace, which a program allocates once; the plain forms have none."""
    if not own:
        return None
    import gemm_reduce_fusion_gb300 as tp
    return tp.workspace(getattr(tp, "TP_OP_" + op), *sizes)


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gemm_reduce_fusion_gb300 as tp
    c, op = s["case"], s["case"]["op"]
    if op in ("norm_fwd", "norm_bwd"):
        kind = {RMS: tp.TP_NORM_RMS, LAYER: tp.TP_NORM_LAYER, "none": tp.TP_NORM_NONE}
        how = dict(post=kind[c["post"]], w_post=s["w_post"], b_post=s["b_post"], pre=kind[c["pre"]], w_pre=s["w_pre"],
                   gate=s["gate"], alpha=s["alpha"])
        if op == "norm_fwd":
            tp.tp_block_norm_fwd(s["x"], s["z"], s["y"], s["n"], b_pre=s["b_pre"], **how)
            return s["y"], s["n"]
        grads = {k: s[k] for k in ("dw_post", "db_post", "dw_pre", "db_pre", "dgate")}
        tp.tp_block_norm_bwd(s["z"], s["y"], s["dn"], s["dy"], s["dx"], s["dz"], s["ws"], **grads, **how)
        return s["dx"], s["dz"], grads
    if op == "ckpt":
        tp.tp_ckpt_pack(s["x"], s["q"], s["e"])
        tp.tp_ckpt_unpack(s["q"], s["e"], s["y"], epi=tp.TP_EPI_GELU if c["gelu"] else tp.TP_EPI_NONE)
        return s["y"]
    if op == "row_bwd_ckpt":
        tp.tp_row_linear_bwd_ckpt(s["q"], s["e"], s["w"], s["dy"][0], s["dx"], s["dw"], s["ws"], epi=tp.TP_EPI_DGELU)
        return s["dx"], s["dw"]
    if op == "col_bwd_ckpt":
        tp.tp_col_linear_bwd_ckpt(s["q"][0], s["e"][0], s["w"], s["dy"], s["dx"][0], s["dw"], s["ws"])
        return s["dx"], s["dw"]
    if op == "row_w4":
        tp.tp_row_linear_fwd_w4(s["x"], s["q"], s["s"], s["out"][0], s["ws"], group=c["G"])
    else:
        tp.tp_col_linear_fwd_w4(s["x"][0], s["q"], s["s"], s["out"], s["ws"], group=c["G"],
                                epi=tp.TP_EPI_GELU if c["gelu"] else tp.TP_EPI_NONE)
    return s["out"]


EPS = 1e-5


def _gelu(x):
    return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))


def _gelu_prime(x):
    return 0.5 * (1 + torch.erf(x * 0.5 ** 0.5)) + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))


def _hat(v, kind):
    """The normalised rows of v and the reciprocal of their deviation."""
    if kind == LAYER:
        v = v - v.mean(1, keepdim=True)
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * r, r


def _norm(v, kind, w, b):
    if kind == "none":
        return v
    n = _hat(v, kind)[0] * w.float()
    return n if b is None else n + b.float()


def _norm_back(u, hat, r, kind):
    """The gradient of v, where u is the gradient of hat(v)."""
    d = u - hat * (u * hat).mean(1, keepdim=True)
    return r * (d - u.mean(1, keepdim=True) if kind == LAYER else d)


def _w4_plain(q, s, K, N, G):
    """The weights [K, N] that q and s stand for, in 32 bits.

    q [a, b, 1024 bytes] holds columns 32 a .. and rows 64 b .. as 256 words
    in the order (f, i, t, d, j), nibble 4 v + 2 u + r of a word at
    k = 64 b + 32 d + 8 t + 4 j + 2 u + v, n = 32 a + 16 f + 8 r + i; a nibble
    stands for itself minus 8, times the scale of its column and group of G
    rows; s [a, group, 32] has column 32 a + 16 f + 8 r + i at 16 f + 2 i + r."""
    a, b = q.shape[:2]
    word = q.view(torch.int32).view(a, b, 2, 8, 4, 2, 2, 1)
    n = (word >> torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)) & 15
    n = n.view(a, b, 2, 8, 4, 2, 2, 2, 2, 2).permute(1, 5, 4, 6, 8, 7, 0, 2, 9, 3).reshape(b * 64, a * 32)[:K, :N]
    s = s.float().view(a, -1, 2, 8, 2).permute(1, 0, 2, 4, 3).reshape(-1, a * 32)[:, :N]
    return (n - 8).float() * s.repeat_interleave(G, 0)[:K]


def _run_plain(s):
    c, op, p = s["case"], s["case"]["op"], s["case"]["p"]
    bf = torch.bfloat16
    if op in ("norm_fwd", "norm_bwd"):
        M, h = c["M"], c["h"]
        z = torch.cat(s["z"]).float()
        gate = s["gate"].float().repeat_interleave(M // c["gate"], 0) if c["gate"] > 1 else s["gate"].float() if c["gate"] else None
        if op == "norm_fwd":
            o = s["alpha"] * _norm(z, c["post"], s["w_post"], s["b_post"])
            y = torch.cat(s["x"]).float() + (o if gate is None else o * gate)
            n = _norm(y, c["pre"], s["w_pre"], s["b_pre"])
            return list(y.to(s["x"][0].dtype).chunk(p)), list(n.to(bf).chunk(p))
        y, dn, dy = torch.cat(s["y"]).float(), torch.cat(s["dn"]).float(), torch.cat(s["dy"]).float()
        hat, r = _hat(y, c["pre"])
        dx = dy + _norm_back(dn * s["w_pre"].float(), hat, r, c["pre"])
        grads = dict.fromkeys(("dw_post", "db_post", "dw_pre", "db_pre", "dgate"))
        grads["dw_pre"] = (dn * hat).sum(0)
        if c["pre"] == LAYER:
            grads["db_pre"] = dn.sum(0)
        if c["gate"]:
            grads["dgate"] = (s["alpha"] * dx * _norm(z, c["post"], s["w_post"], s["b_post"])).view(c["gate"], -1, h).sum(1)
        do = s["alpha"] * dx if gate is None else s["alpha"] * dx * gate
        dz = do
        if c["post"] != "none":
            hat, r = _hat(z, c["post"])
            grads["dw_post"] = (do * hat).sum(0)
            if c["post"] == LAYER:
                grads["db_post"] = do.sum(0)
            dz = _norm_back(do * s["w_post"].float(), hat, r, c["post"])
        return list(dx.to(s["y"][0].dtype).chunk(p)), list(dz.to(bf).chunk(p)), grads
    if op == "ckpt":
        v = [_unpack_plain(*_pack_plain(x)) for x in s["x"]]
        return [(_gelu(x) if c["gelu"] else x).to(bf) for x in v]
    if op == "row_bwd_ckpt":
        h = [_unpack_plain(q, e) for q, e in zip(s["q"], s["e"])]
        dy = s["dy"][0].float()
        dx = [(dy @ w.float().t() * _gelu_prime(v)).to(bf) for w, v in zip(s["w"], h)]
        return dx, [(_gelu(v).t() @ dy).to(bf) for v in h]
    if op == "col_bwd_ckpt":
        x = _unpack_plain(s["q"][0], s["e"][0])
        dx = torch.cat(s["dy"], 1).float() @ torch.cat(s["w"], 1).float().t()
        return [dx.to(bf)], [(x.t() @ dy.float()).to(bf) for dy in s["dy"]]
    w = [_w4_plain(q, k, c["K"], c["N"], c["G"]) for q, k in zip(s["q"], s["s"])]
    dtype = torch.float32 if c["f32"] else bf
    if op == "row_w4":
        return [(torch.cat(s["x"], 1).float() @ torch.cat(w)).to(dtype)]
    y = [s["x"][0].float() @ a for a in w]
    return [(_gelu(v) if c["gelu"] else v).to(dtype) for v in y]


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    """What run returns for these inputs, row by row from the definitions, in 64 bits."""
    c, s, p = case, prepare(case, seed), case["p"]
    D = torch.float64

    def moments(v, kind):
        mu = v.sum(-1) / v.shape[-1] if kind == LAYER else torch.zeros(v.shape[0], dtype=D, device=v.device)
        var = ((v - mu[:, None]) ** 2).sum(-1) / v.shape[-1]
        return mu[:, None], (var + EPS).rsqrt()[:, None]

    def two_to(e):  # by its bits: pow(2, e) may be off in the last one, and halves would then round the other way
        return ((e.to(torch.int64) + 1023) << 52).view(D)

    def phi(v):
        return torch.special.erfc(-v / math.sqrt(2)) / 2

    def saved(q, e):
        group = torch.arange(q.shape[1], device=q.device) // 32
        v = q.to(D) * two_to(e.to(torch.int64) - 126)[:, group]
        return torch.where(e[:, group] == 255, torch.full_like(v, math.nan), v)

    if c["op"] in ("norm_fwd", "norm_bwd"):
        ones, zeros = torch.ones(c["h"], dtype=D, device="cuda"), torch.zeros(c["h"], dtype=D, device="cuda")
        vec = lambda k, other: other if s[k] is None else s[k].to(D)  # noqa: E731
        wq, bq, wp, bp = vec("w_post", ones), vec("b_post", zeros), vec("w_pre", ones), vec("b_pre", zeros)
        m, per = c["M"] // p, c["M"] // max(1, c["gate"])
        first, second, grads = [], [], {}
        sums = {k: torch.zeros(c["h"], dtype=D, device="cuda") for k in ("dw_post", "db_post", "dw_pre", "db_pre")}
        dgate = torch.zeros((max(1, c["gate"]), c["h"]), dtype=D, device="cuda")
        for k in range(p):
            z = s["z"][k].to(D)
            at = (torch.arange(m, device="cuda") + k * m) // per
            g = s["alpha"] * (s["gate"].to(D)[at] if c["gate"] else torch.ones_like(z))
            mu, r = moments(z, c["post"]) if c["post"] != "none" else (0, 1)
            zh = (z - mu) * r
            o = zh * wq + bq
            if c["op"] == "norm_fwd":
                y = s["x"][k].to(D) + g * o
                mu, r = moments(y, c["pre"])
                first.append(y)
                second.append((y - mu) * r * wp + bp)
                continue
            y, dn = s["y"][k].to(D), s["dn"][k].to(D)
            my, ry = moments(y, c["pre"])
            yh, t = (y - my) * ry, dn * wp
            dx = s["dy"][k].to(D) + ry * (t - (t.mean(1, keepdim=True) if c["pre"] == LAYER else 0) - yh * (t * yh).mean(1, keepdim=True))
            sums["dw_pre"] += (dn * yh).sum(0)
            sums["db_pre"] += dn.sum(0)
            dgate.index_add_(0, at, s["alpha"] * dx * o)
            t = g * dx
            sums["dw_post"] += (t * zh).sum(0)
            sums["db_post"] += t.sum(0)
            t = t * wq
            if c["post"] != "none":
                t = r * (t - (t.mean(1, keepdim=True) if c["post"] == LAYER else 0) - zh * (t * zh).mean(1, keepdim=True))
            first.append(dx)
            second.append(t)
        if c["op"] == "norm_fwd":
            return first, second
        grads = {k: None if s[k[1:]] is None else v for k, v in sums.items()}
        grads["dgate"] = dgate if c["gate"] else None
        return first, second, grads
    if c["op"] == "ckpt":
        out = []
        for x in s["x"]:
            M, N = x.shape
            v = torch.nn.functional.pad(x.to(D), (0, -N % 32)).view(M, -1, 32)
            top = v.abs().amax(2)
            e = torch.ceil(torch.log2(top / 127)).clamp(min=-126)
            e = torch.where(top > 127 * two_to(e), e + 1, e)
            e = torch.where((top <= 127 * two_to(e - 1)) & (e > -126), e - 1, e)
            step = two_to(e)[..., None]
            v = (torch.round(v / step) * step).view(M, -1)[:, :N]
            out.append(v * phi(v) if c["gelu"] else v)
        return out
    if c["op"] in ("row_bwd_ckpt", "col_bwd_ckpt"):
        v = [saved(q, e) for q, e in zip(s["q"], s["e"])]
        w, dy = [a.to(D) for a in s["w"]], [a.to(D) for a in s["dy"]]
        if c["op"] == "col_bwd_ckpt":
            return [sum(b @ a.t() for a, b in zip(w, dy))], [v[0].t() @ b for b in dy]
        slope = [phi(h) + h * torch.exp(-h * h / 2) / math.sqrt(2 * math.pi) for h in v]
        return [dy[0] @ a.t() * k for a, k in zip(w, slope)], [(h * phi(h)).t() @ dy[0] for h in v]
    K, N, G = c["K"], c["N"], c["G"]
    k, n = torch.arange(K, device="cuda")[:, None], torch.arange(N, device="cuda")[None, :]
    # byte 2 * (16-byte lane word ...) of each weight, straight from its row and column
    word = ((n // 16 % 2 * 8 + n % 8) * 4 + k // 8 % 4) * 4 + k // 32 % 2 * 2 + k // 4 % 2
    nibble = 4 * (k % 2) + 2 * (k // 2 % 2) + n // 8 % 2
    place = (n // 32 * -(-K // 64) + k // 64) * 1024 + word * 4 + nibble // 2
    lane = (n // 32 * -(-K // G) + k // G) * 32 + n // 16 % 2 * 16 + n % 8 * 2 + n // 8 % 2
    w = []
    for q, sc in zip(s["q"], s["s"]):
        v = torch.where(nibble % 2 == 1, q.view(-1)[place] >> 4, q.view(-1)[place] & 15)
        w.append((v.to(D) - 8) * sc.view(-1)[lane].to(D))
    if c["op"] == "row_w4":
        return [sum(x.to(D) @ a for x, a in zip(s["x"], w))]
    y = [s["x"][0].to(D) @ a for a in w]
    return [v * phi(v) if c["gelu"] else v for v in y]
