"""Plain 64-bit implementations of the operators around the sharded Linear,
for their tests: written from the definitions, on the CPU, with none of the
library's code."""
import torch

D = torch.float64


def gelu(v):
    return v * torch.special.erfc(-v / 2 ** 0.5) / 2


def gelu_prime(v):
    return torch.special.erfc(-v / 2 ** 0.5) / 2 + v * torch.exp(-v * v / 2) / (2 * torch.pi) ** 0.5


# ------------------------------------------------------------------ norms

def hat(v, kind, eps):
    """Normalised rows and 1 / deviation; kind "none", "rms" or "layer"."""
    if kind == "none":
        return v, torch.ones((v.shape[0], 1), dtype=D)
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    return v * r, r


def norm(v, kind, w, b, eps):
    n = hat(v, kind, eps)[0]
    n = n if w is None else n * w
    return n if b is None else n + b


def norm_back(u, v, kind, eps):
    """Gradient of v given that of hat(v)."""
    if kind == "none":
        return u
    h, r = hat(v, kind, eps)
    g = u - h * (u * h).mean(1, keepdim=True)
    if kind == "layer":
        g = g - u.mean(1, keepdim=True)
    return r * g


def rows_of_gate(gate, M):
    return None if gate is None else gate.repeat_interleave(M // gate.shape[0], 0)


def block_fwd(x, z, d):
    """(y, n) of full [M, h] tensors; d: post, pre, w_post, b_post, w_pre, b_pre, gate, alpha, eps."""
    y = x
    if z is not None:
        o = norm(z, d["post"], d["w_post"], d["b_post"], d["eps"])
        g = rows_of_gate(d["gate"], x.shape[0])
        y = x + d["alpha"] * (o if g is None else o * g)
    return y, norm(y, d["pre"], d["w_pre"], d["b_pre"], d["eps"])


def block_bwd(y, z, dn, dy, d):
    """Gradients as a dict, and for each column sum the sum of its terms' magnitudes under "|name|"."""
    M = (y if y is not None else dy).shape[0]
    out = {}
    dx = torch.zeros_like(y if y is not None else dy) if dy is None else dy.clone()

    def total(name, terms):
        out[name], out["|" + name + "|"] = terms.sum(0), terms.abs().sum(0)

    if dn is not None:
        h = hat(y, d["pre"], d["eps"])[0]
        total("dw_pre", dn * h)
        total("db_pre", dn)
        dx = dx + norm_back(dn if d["w_pre"] is None else dn * d["w_pre"], y, d["pre"], d["eps"])
    out["dx"] = dx
    if z is not None:
        g = rows_of_gate(d["gate"], M)
        if g is not None:
            t = d["alpha"] * dx * norm(z, d["post"], d["w_post"], d["b_post"], d["eps"])
            t = t.view(d["gate"].shape[0], -1, t.shape[1])
            out["dgate"], out["|dgate|"] = t.sum(1), t.abs().sum(1)
        t = d["alpha"] * dx if g is None else d["alpha"] * dx * g
        total("dw_post", t * hat(z, d["post"], d["eps"])[0])
        total("db_post", t)
        out["dz"] = norm_back(t if d["w_post"] is None else t * d["w_post"], z, d["post"], d["eps"])
    return out


# ------------------------------------------------------------------ 8-bit checkpoints

def ckpt_pack(x):
    """(q, e) of x [M, N], group by group with exact arithmetic on 64-bit floats."""
    M, N = x.shape
    G = -(-N // 32)
    q, e = torch.zeros((M, N), dtype=torch.int8), torch.zeros((M, G), dtype=torch.uint8)
    v = x.to(D)
    for c in range(G):
        part = v[:, 32 * c:32 * c + 32]
        bad = ~torch.isfinite(part).all(1)
        top = torch.where(bad, torch.zeros(M, dtype=D), part.abs().amax(1))
        E = torch.full((M,), -126, dtype=torch.int64)
        while True:  # the smallest E with 127 * 2^E >= top
            more = 127 * two_to(E) < top
            if not more.any():
                break
            E = E + more.to(torch.int64)
        r = torch.round(part / two_to(E)[:, None])  # a division by a power of two: exact
        q[:, 32 * c:32 * c + 32] = torch.where(bad[:, None], torch.zeros_like(r), r).to(torch.int8)
        e[:, c] = torch.where(bad, torch.full_like(E, 255), E + 126).to(torch.uint8)
    return q, e


def two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(D)


def ckpt_value(q, e):
    g = torch.arange(q.shape[1]) // 32
    v = q.to(D) * two_to(e.to(torch.int64) - 126)[:, g]
    return torch.where(e[:, g] == 255, torch.full_like(v, float("nan")), v)


# ------------------------------------------------------------------ 4-bit weights

def w4_place(K, N):
    """For k, n of a [K, N] weight: index of its 32-bit word and of its nibble in it."""
    k, n = torch.arange(K)[:, None], torch.arange(N)[None, :]
    a, f, r, i = n // 32, n // 16 % 2, n // 8 % 2, n % 8
    b, d, t, j, u, v = k // 64, k // 32 % 2, k // 8 % 4, k // 4 % 2, k // 2 % 2, k % 2
    word = (a * -(-K // 64) + b) * 256 + f * 128 + i * 16 + t * 4 + d * 2 + j
    return word, 4 * v + 2 * u + r


def w4_scale_place(K, N, G):
    k, n = torch.arange(K)[:, None], torch.arange(N)[None, :]
    return (n // 32 * -(-K // G) + k // G) * 32 + n // 16 % 2 * 16 + n % 8 * 2 + n // 8 % 2


def w4_value(q, s, K, N, G):
    word, nib = w4_place(K, N)
    words = q.cpu().contiguous().view(torch.int32).view(-1).to(torch.int64)
    v = (words[word] >> (4 * nib)) & 15
    return (v.to(D) - 8) * s.cpu().to(D).view(-1)[w4_scale_place(K, N, G)]


def w4_quant(w, G):
    """Whole numbers in 0..15 and bf16 scales [ceil(K/G), N] of bf16 weights w [K, N]."""
    K, N = w.shape
    v = w.to(D)
    s = torch.stack([v[g:g + G].abs().amax(0) for g in range(0, K, G)])
    s = torch.where(torch.isfinite(s), s / 7, torch.full_like(s, float("nan"))).to(torch.bfloat16)
    full = s.to(D).repeat_interleave(G, 0)[:K]
    r = torch.where(full > 0, torch.round(v / torch.where(full > 0, full, torch.ones_like(full))), torch.zeros_like(v))
    return (r.clamp(-7, 7) + 8).to(torch.int64), s
