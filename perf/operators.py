"""The training-side operators of a DiT block's norm / modulation path, as cases to measure.

Four groups that run next to each other in one block:

* ``layer_norm``                 affine LayerNorm, y = (x - mean) * rstd * w + b
* ``layer_norm_backward``        its gradients dx, dw, db (the statistics come from x again)
* ``ln_modulate_backward``       the gradients of LN(x) * (1 + scale) + shift, with scale and shift
                                 shared by a whole sample, or one row of each for every token
* ``dropout``, ``dropout_gate_add`` and ``dropout_gate_add_backward``
                                 x + gate * drop(y); the mask is a function of (seed, counter, row,
                                 column) and is never stored
* ``rope_axes``                  the rotation of Q and K by positions on several axes (time, height,
                                 width); its backward pass is the rotation by the opposite angle

``own`` false computes them with elementary torch operations, ``own`` true calls this repository's
package.  ``exact`` gives the same outputs in binary64.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
_mbx = None


def _lib():
    global _mbx
    if _mbx is None:
        import modulation_bit_exact_gb300 as m
        _mbx = m
    return _mbx


# ---------------------------------------------------------------- cases


def listed():
    return [
        # affine LayerNorm of one short text prompt: launch latency
        dict(name="ln_text_77x1024", op="ln", rows=77, dim=1024, dtype="bf16", pdtype="bf16"),
        # the affine norm before cross-attention in a video DiT block (21 x 30 x 52 latent tokens)
        dict(name="ln_video_32760x5120", op="ln", rows=32760, dim=5120, dtype="bf16", pdtype="bf16"),
        # a float32 encoder of odd width, rows that start at no 16-byte boundary
        dict(name="ln_f32_4099x1931", op="ln", rows=4099, dim=1931, dtype="f32", pdtype="f32"),
        # affine LayerNorm's gradients for many short rows: the weight's gradient sums 65536 rows
        dict(name="lnb_65536x1024", op="lnb", rows=65536, dim=1024, dtype="bf16", pdtype="f32", res=False),
        # AdaLN gradients of an image DiT block, one modulation row a sample, added to the residual
        # stream's gradient
        dict(name="modb_image_2x4352x4096", op="modb", rows=8704, dim=4096, mod_rows=2, dtype="bf16",
             pdtype="bf16", res=True),
        # AdaLN gradients of a video DiT block with one modulation row a token: the largest call
        dict(name="modb_video_token_32760x5120", op="modb", rows=32760, dim=5120, mod_rows=32760, dtype="bf16",
             pdtype="bf16", res=False),
        # gated residual with dropout on a small batch: launch latency
        dict(name="drop_small_2x256x512", op="dropgate", rows=512, dim=512, mod_rows=2, dtype="bf16",
             pdtype="bf16", p=0.1),
        # the same over a video sequence
        dict(name="drop_video_32760x5120", op="dropgate", rows=32760, dim=5120, mod_rows=1, dtype="bf16",
             pdtype="bf16", p=0.1),
        # its gradients for an image batch: dy, and the gate's gradient summed over each sample
        dict(name="dropb_image_2x4352x4096", op="dropgateb", rows=8704, dim=4096, mod_rows=2, dtype="bf16",
             pdtype="bf16", p=0.1),
        # plain dropout of a float32 activation of odd width
        dict(name="dropout_f32_4096x2731", op="dropout", rows=4096, dim=2731, dtype="f32", p=0.25),
        # Q and K of a video DiT block: three axes over a 21 x 30 x 52 grid
        dict(name="rope_video_32760x40x128", op="rope", batch=1, tokens=32760, qheads=40, kheads=40, hd=128,
             a0=44, a1=42, a2=42, dtype="bf16", interleaved=True, inverse=False, merged=False, ptype="i32"),
        # one new token for each of eight sequences, grouped K heads, read from the merged QKV rows
        dict(name="rope_token_8x32x8x128", op="rope", batch=8, tokens=1, qheads=32, kheads=8, hd=128,
             a0=32, a1=48, a2=48, dtype="bf16", interleaved=False, inverse=False, merged=True, ptype="i32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "lnb", "modb", "modb", "dropgate", "dropgateb", "dropout", "rope", "rope"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    most = 120_000_000 if dtype == "bf16" else 60_000_000
    if op == "rope":
        hd = rng.choice([64, 128, 128, 256, 80])
        kheads = rng.choice([1, 2, 8, 24, 40])
        qheads = kheads * rng.choice([1, 1, 4])
        batch = rng.choice([1, 1, 2, 5])
        tokens = _log(rng, 1, max(2, min(65536, most // (batch * (qheads + kheads) * hd))))
        part = hd // 2 if rng.random() < 0.2 else hd  # some models rotate only the first part of a head
        a0 = 2 * rng.randint(1, part // 8)
        a1 = 2 * ((part - a0) // 4)
        return dict(op=op, batch=batch, tokens=tokens, qheads=qheads, kheads=kheads, hd=hd, a0=a0, a1=a1,
                    a2=part - a0 - a1, dtype=dtype, interleaved=rng.random() < 0.6, inverse=rng.random() < 0.5,
                    merged=rng.random() < 0.5, ptype=rng.choice(["i32", "f32"]))
    dim = _log(rng, 64, 8192)
    if rng.random() < 0.75:
        dim = max(64, dim // 8 * 8)
    rows = _log(rng, 1, max(2, min(65536, most // dim)))
    case = dict(op=op, rows=rows, dim=dim, dtype=dtype)
    if op != "dropout":
        case["pdtype"] = "f32" if dtype == "f32" else rng.choice(["bf16", "bf16", "f32"])
    if op in ("modb", "dropgate", "dropgateb"):
        m = rng.choice([1, 2, 4, rows])  # shared by the batch, one a sample, one a token
        case["rows"] = rows = max(1, rows // m) * m
        case["mod_rows"] = m
    if op in ("lnb", "modb"):
        case["res"] = rng.random() < 0.5
    if op in ("dropgate", "dropgateb", "dropout"):
        case["p"] = rng.choice([0.0, 0.1, 0.1, 0.25, 0.5])
    return case


# ---------------------------------------------------------------- inputs


def _normal(g, shape, dt, std=1.0, mean=0.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).add_(mean).to(dt)


def _activations(g, rows, dim, dt):
    """N(0, 1) with 1 % of the elements x 20 (the outlier channels of trained blocks) and a mean of
    each row's own."""
    x = torch.randn((rows, dim), generator=g, device=DEV)
    x = torch.where(torch.rand((rows, dim), generator=g, device=DEV) < 0.01, x * 20.0, x)
    return (x + torch.randn((rows, 1), generator=g, device=DEV) * 0.5).to(dt)


def _positions(case, g):
    """Grid positions (time, height, width) of each token, the batch sharing them; fractional where
    the case's positions are float32 (resolution-scaled grids)."""
    S = case["tokens"]
    if S == 1:  # single new tokens: each sequence has a position of its own, far ones among them
        pos = torch.randint(0, 100_000, (case["batch"], 1, 3), generator=g, device=DEV)
    else:
        w = max(1, int(round((S / 21) ** 0.5 * 1.3)))
        h = max(1, -(-S // (21 * w)))
        i = torch.arange(S, device=DEV)
        first = torch.randint(0, 1000, (1,), generator=g, device=DEV)
        pos = torch.stack([i // (h * w) + first, (i // w) % h, i % w], dim=1)
    if case["ptype"] == "f32":
        return pos.float() * 0.7109375
    return pos.int()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    dt = DT[case["dtype"]]
    if op == "rope":
        B, S, hq, hk, hd = (case[k] for k in ("batch", "tokens", "qheads", "kheads", "hd"))
        if case["merged"]:  # rows of a merged QKV product, K heads as many as V heads
            qkv = _normal(g, (B, S, hq + 2 * hk, hd), dt)
            s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
        else:
            s["q"], s["k"] = _normal(g, (B, S, hq, hd), dt), _normal(g, (B, S, hk, hd), dt)
        s["pos"] = _positions(case, g)
        s["axes"] = (case["a0"], case["a1"], case["a2"])
        # the plan a model keeps: the angle per position of every pair, in radians
        s["freqs"] = torch.cat([
            torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=DEV),
                      torch.arange(0, a, 2, dtype=torch.float64, device=DEV) / -a) for a in s["axes"]])
        return s
    rows, dim = case["rows"], case["dim"]
    pdt = DT[case.get("pdtype", case["dtype"])]
    s["x"] = _activations(g, rows, dim, dt)
    if op == "ln":
        s["weight"], s["bias"] = _normal(g, (dim,), pdt, 0.05, 1.0), _normal(g, (dim,), pdt, 0.1)
    if op in ("lnb", "modb"):
        s["dout"] = _normal(g, (rows, dim), dt, 0.01)
        s["dres"] = _normal(g, (rows, dim), dt, 0.01) if case["res"] else None
        if op == "lnb":
            s["weight"] = _normal(g, (dim,), pdt, 0.05, 1.0)
        else:
            s["scale"] = _normal(g, (case["mod_rows"], dim), pdt, 0.1)
    if op in ("dropgate", "dropgateb"):
        s["gate"] = _normal(g, (case["mod_rows"], dim), pdt, 0.1)
        s["y"] = _normal(g, (rows, dim), dt)
    if op == "dropgateb":
        s["dout"] = s.pop("x")
    if "p" in case:  # the generator's state: a seed and the step's counter
        s["rng"] = torch.tensor([0x5DEECE66D + int(seed), 17 + 1000 * int(seed)], dtype=torch.int64, device=DEV)
    return s


OFFSET = 3  # the layer's own offset of the counter


# ---------------------------------------------------------------- the plain forms


def _by_sample(t, mod_rows):
    return t.reshape(mod_rows, -1, t.shape[-1])


def _mul_hi_lo(const, v):
    """High and low 32 bits of const * v for 32-bit values held in int64."""
    t = (const & 0xFFFF) * v
    u = (const >> 16) * v + (t >> 16)
    return u >> 16, ((u & 0xFFFF) << 16) | (t & 0xFFFF)


def _keep(rows, dim, p, rng, offset):
    """The mask: Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011)
    with the key rng[0] and the counter (column / 4, row, rng[1] + offset); column c uses word c mod 4
    and is kept where that word is at least floor(p * 2^32)."""
    m32 = 0xFFFFFFFF
    nq = -(-dim // 4)
    step = rng[1] + offset
    c0 = torch.arange(nq, device=DEV, dtype=torch.int64).expand(rows, nq)
    c1 = torch.arange(rows, device=DEV, dtype=torch.int64)[:, None].expand(rows, nq)
    c2, c3 = (step & m32).expand(rows, nq), ((step >> 32) & m32).expand(rows, nq)
    k0, k1 = rng[0] & m32, (rng[0] >> 32) & m32
    for _ in range(10):
        h0, l0 = _mul_hi_lo(0xD2511F53, c0)
        h1, l1 = _mul_hi_lo(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    thr = int(math.floor(p * 4294967296.0))
    words = torch.stack([c0, c1, c2, c3], dim=-1).reshape(rows, nq * 4)[:, :dim]
    return words >= thr


def _xhat(x):
    xf = x.float()
    xc = xf - xf.mean(dim=-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(xc.square().mean(dim=-1, keepdim=True) + EPS)
    return xc * rstd, rstd


def _ln_grads(s, factor, mod_rows):
    """dx, and the gradients of the factor and of the shift (summed over each modulation row)."""
    xhat, rstd = _xhat(s["x"])
    dy = s["dout"].float()
    gy = (_by_sample(dy, mod_rows) * factor[:, None]).reshape(dy.shape)
    dx = rstd * (gy - gy.mean(dim=-1, keepdim=True) - xhat * (gy * xhat).mean(dim=-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    dfactor = _by_sample(dy * xhat, mod_rows).sum(dim=1)
    dshift = _by_sample(dy, mod_rows).sum(dim=1)
    return dx.to(s["x"].dtype), dfactor, dshift


def _rope_plain(t, pos, freqs, axes, interleaved, inverse):
    B, S, H, hd = t.shape
    n = sum(axes) // 2
    axis_of = [i for i, a in enumerate(axes) for _ in range(a // 2)]
    ang = pos.double().reshape(-1, S, len(axes))[:, :, axis_of] * freqs  # [1 or B, S, n], 64 bits
    c, sn = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]
    sn = -sn if inverse else sn
    f = t.float()
    a, b = (f[..., 0:2 * n:2], f[..., 1:2 * n:2]) if interleaved else (f[..., :n], f[..., n:2 * n])
    o0, o1 = a * c - b * sn, a * sn + b * c
    o = torch.stack([o0, o1], dim=-1).flatten(-2) if interleaved else torch.cat([o0, o1], dim=-1)
    return torch.cat([o, f[..., 2 * n:]], dim=-1).to(t.dtype)


def _run_plain(s):
    op = s["op"]
    if op == "rope":
        return tuple(_rope_plain(s[k], s["pos"], s["freqs"], s["axes"], s["interleaved"], s["inverse"])
                     for k in ("q", "k"))
    if op == "ln":
        return (_xhat(s["x"])[0] * s["weight"].float() + s["bias"].float()).to(s["x"].dtype)
    if op == "lnb":
        dx, dw, db = _ln_grads(s, s["weight"].float()[None], 1)
        return dx, dw[0].to(s["weight"].dtype), db[0].to(s["weight"].dtype)
    if op == "modb":
        dx, dsc, dsh = _ln_grads(s, 1.0 + s["scale"].float(), s["mod_rows"])
        return dx, dsc.to(s["scale"].dtype), dsh.to(s["scale"].dtype)
    keep = _keep(s["rows"], s["dim"], s["p"], s["rng"], OFFSET)
    inv = 1.0 / (1.0 - s["p"])
    if op == "dropout":
        return torch.where(keep, s["x"].float() * inv, 0.0).to(s["x"].dtype)
    m = s["mod_rows"]
    gate = s["gate"].float()[:, None]
    y, kept = _by_sample(s["y"].float() * inv, m), _by_sample(keep, m)
    if op == "dropgate":
        x = _by_sample(s["x"].float(), m)
        return torch.where(kept, x + gate * y, x).reshape(s["x"].shape).to(s["x"].dtype)
    do = _by_sample(s["dout"].float(), m)
    dy = torch.where(kept, do * gate * inv, 0.0).reshape(s["y"].shape).to(s["y"].dtype)
    return dy, torch.where(kept, do * y, 0.0).sum(dim=1).to(s["gate"].dtype)


# ---------------------------------------------------------------- one pass


def _run_own(s):
    m = _lib()
    op = s["op"]
    if op == "rope":
        return m.rope_axes(s["q"], s["k"], s["pos"], s["freqs"], s["axes"], interleaved=s["interleaved"],
                           inverse=s["inverse"])
    if op == "ln":
        return m.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
    if op == "lnb":
        return m.layer_norm_backward(s["dout"], s["x"], s["weight"], eps=EPS, dresidual=s["dres"])
    if op == "modb":
        return m.ln_modulate_backward(s["dout"], s["x"], s["scale"], eps=EPS, dresidual=s["dres"])
    if op == "dropout":
        return m.dropout(s["x"], s["p"], s["rng"], offset=OFFSET)
    if op == "dropgate":
        return m.dropout_gate_add(s["x"], s["gate"], s["y"], s["p"], s["rng"], offset=OFFSET)
    return m.dropout_gate_add_backward(s["dout"], s["gate"], s["y"], s["p"], s["rng"], offset=OFFSET)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- binary64


def _exact_ln(s, grads):
    """LayerNorm in binary64 by row blocks; the gradients by differentiating the definition."""
    rows, dim = s["x"].shape
    m = s.get("mod_rows", 1)
    seq = rows // m
    if "scale" in s:
        factor = s["scale"].double() + 1.0
    else:
        factor = s["weight"].double().reshape(1, dim)
    shift = s["bias"].double().reshape(1, dim) if "bias" in s else torch.zeros_like(factor)
    outs, dfac, dsh = [], torch.zeros_like(factor), torch.zeros_like(factor)
    block = max(1, (1 << 23) // dim)
    for lo in range(0, rows, block):
        hi = min(rows, lo + block)
        ma, mb = lo // seq, (hi - 1) // seq + 1
        which = torch.arange(lo, hi, device=DEV) // seq - ma
        x = s["x"][lo:hi].double().requires_grad_(grads)
        f = factor[ma:mb][which].requires_grad_(grads)  # one row of each for every row of x
        b = shift[ma:mb][which].requires_grad_(grads)
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        out = (x - mean) * (var + EPS) ** -0.5 * f + b
        if not grads:
            outs.append(out)
            continue
        gx, gf, gb = torch.autograd.grad(out, (x, f, b), s["dout"][lo:hi].double())
        outs.append(gx if s["dres"] is None else gx + s["dres"][lo:hi].double())
        dfac.index_add_(0, which + ma, gf)
        dsh.index_add_(0, which + ma, gb)
    y = torch.cat(outs)
    if not grads:
        return y
    if "scale" in s:
        return y, dfac, dsh
    return y, dfac[0], dsh[0]


def _exact_keep(s, lo, hi):
    """The mask of rows lo..hi with wrapping 64-bit products."""
    dim = s["dim"]
    key, step = s["rng"].tolist()
    step += OFFSET
    quad = torch.arange((dim + 3) // 4, device=DEV)
    row = torch.arange(lo, hi, device=DEV)
    w = [quad.repeat(hi - lo, 1), row[:, None].repeat(1, len(quad)),
         torch.full((hi - lo, len(quad)), step % 2 ** 32, device=DEV),
         torch.full((hi - lo, len(quad)), (step >> 32) % 2 ** 32, device=DEV)]
    ka, kb = key % 2 ** 32, (key >> 32) % 2 ** 32
    for r in range(10):
        pa, pb = w[0] * 0xD2511F53, w[2] * 0xCD9E8D57  # modulo 2^64
        w = [((pb >> 32) & 0xFFFFFFFF) ^ w[1] ^ ((ka + r * 0x9E3779B9) % 2 ** 32), pb & 0xFFFFFFFF,
             ((pa >> 32) & 0xFFFFFFFF) ^ w[3] ^ ((kb + r * 0xBB67AE85) % 2 ** 32), pa & 0xFFFFFFFF]
    keep = torch.empty((hi - lo, 4 * len(quad)), dtype=torch.bool, device=DEV)
    for i in range(4):
        keep[:, i::4] = w[i] >= int(s["p"] * 2.0 ** 32)
    return keep[:, :dim]


def _exact_dropout(s):
    op, rows, dim = s["op"], s["rows"], s["dim"]
    m = s.get("mod_rows", 1)
    seq = rows // m
    outs = []
    dgate = torch.zeros((m, dim), dtype=torch.float64, device=DEV)
    block = max(1, (1 << 23) // dim)
    for lo in range(0, rows, block):
        hi = min(rows, lo + block)
        mask = _exact_keep(s, lo, hi).double() / (1.0 - s["p"])
        which = torch.arange(lo, hi, device=DEV) // seq
        if op == "dropout":
            outs.append(s["x"][lo:hi].double() * mask)
        elif op == "dropgate":
            outs.append(s["x"][lo:hi].double() + s["gate"].double()[which] * s["y"][lo:hi].double() * mask)
        else:
            do = s["dout"][lo:hi].double()
            outs.append(do * mask * s["gate"].double()[which])
            dgate.index_add_(0, which, do * mask * s["y"][lo:hi].double())
    y = torch.cat(outs)
    return (y, dgate) if op == "dropgateb" else y


def _exact_rope(t, s):
    """Each pair as a complex number times e^(i * angle), or its conjugate."""
    B, S, H, hd = t.shape
    pairs, first = [], 0
    n = sum(s["axes"]) // 2
    pos = s["pos"].double().reshape(-1, S, 3)
    turn = torch.empty((pos.shape[0], S, n), dtype=torch.complex128, device=DEV)
    for i, a in enumerate(s["axes"]):
        for j in range(a // 2):
            ang = pos[:, :, i] * 10000.0 ** (-2.0 * j / a)
            turn[:, :, first + j] = torch.complex(torch.cos(ang), torch.sin(ang))
        first += a // 2
    if s["inverse"]:
        turn = turn.conj().resolve_conj()
    d = t.double()
    if s["interleaved"]:
        z = torch.view_as_complex(d[..., :2 * n].reshape(B, S, H, n, 2))
    else:
        z = torch.complex(d[..., :n].contiguous(), d[..., n:2 * n].contiguous())
    z = z * turn[:, :, None]
    out = d.clone()
    if s["interleaved"]:
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = z.real, z.imag
    else:
        out[..., :n], out[..., n:2 * n] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return tuple(_exact_rope(s[k], s) for k in ("q", "k"))
    if case["op"] == "ln":
        return _exact_ln(s, False)
    if case["op"] in ("lnb", "modb"):
        return _exact_ln(s, True)
    return _exact_dropout(s)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    e = 4 if case["dtype"] == "f32" else 2
    if op == "rope":
        tokens = case["batch"] * case["tokens"]
        n = tokens * (case["qheads"] + case["kheads"]) * case["hd"]
        pos_rows = tokens if case["tokens"] == 1 else case["tokens"]
        pairs = (case["a0"] + case["a1"] + case["a2"]) // 2
        return {"bytes": 2 * n * e + pos_rows * 12 + pairs * 8, "flops": 3 * n}
    n = case["rows"] * case["dim"]
    pe = 4 if case.get("pdtype") == "f32" else 2
    params = case.get("mod_rows", 1) * case["dim"] * pe
    if op == "ln":
        return {"bytes": 2 * n * e + 2 * params, "flops": 8 * n}
    if op in ("lnb", "modb"):
        return {"bytes": (3 + bool(case["res"])) * n * e + 3 * params, "flops": 17 * n}
    if op == "dropout":
        return {"bytes": 2 * n * e + 16, "flops": 2 * n}
    return {"bytes": 3 * n * e + (2 if op == "dropgateb" else 1) * params + 16, "flops": 4 * n}
