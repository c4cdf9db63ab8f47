"""Operators around a DiT block's Q/K heads and its modulation vectors, as cases to measure.

* ``qk_norm_rope``            RMSNorm of every head of Q and K, a weight for each, and the rotation by
                              positions on several axes, in one pass
* ``qk_norm_rope_backward``   its gradients dq, dk, dwq, dwk
* ``linear_nvfp4``            out = a(x) W^T + bias with W in 4 bits (E2M1 values, one E4M3 scale for 16
                              of them, a global scale) for a few rows x, a the identity or SiLU: the
                              projection that makes a block's scale, shift and gate from the time embedding

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
        # Q and K of an image DiT block with guidance, read from the merged QKV product
        dict(name="qkn_image_2x4352x24x128", op="qkn", batch=2, tokens=4352, qheads=24, kheads=24, hd=128,
             a0=16, a1=56, a2=56, dtype="bf16", wdtype="bf16", interleaved=True, merged=True, ptype="i32"),
        # the same of a video DiT block: 21 x 30 x 52 latent tokens of 40 heads
        dict(name="qkn_video_32760x40x128", op="qkn", batch=1, tokens=32760, qheads=40, kheads=40, hd=128,
             a0=44, a1=42, a2=42, dtype="bf16", wdtype="bf16", interleaved=True, merged=False, ptype="i32"),
        # one new token for each of 24 sequences, grouped K heads: launch latency
        dict(name="qkn_token_24x32x8x128", op="qkn", batch=24, tokens=1, qheads=32, kheads=8, hd=128,
             a0=32, a1=48, a2=48, dtype="bf16", wdtype="f32", interleaved=False, merged=True, ptype="i32"),
        # a float32 encoder: heads of 80, of which 40 elements turn, at resolution-scaled positions
        dict(name="qkn_f32_3x1213x16x80", op="qkn", batch=3, tokens=1213, qheads=16, kheads=4, hd=80,
             a0=8, a1=16, a2=16, dtype="f32", wdtype="f32", interleaved=False, merged=False, ptype="f32"),
        # the gradients of the first case
        dict(name="qknb_image_2x4352x24x128", op="qknb", batch=2, tokens=4352, qheads=24, kheads=24, hd=128,
             a0=16, a1=56, a2=56, dtype="bf16", wdtype="bf16", interleaved=True, merged=True, ptype="i32"),
        # the gradients of the second: the largest call
        dict(name="qknb_video_32760x40x128", op="qknb", batch=1, tokens=32760, qheads=40, kheads=40, hd=128,
             a0=44, a1=42, a2=42, dtype="bf16", wdtype="f32", interleaved=True, merged=False, ptype="i32"),
        # gradients of a short text sequence, heads of 64 in halves, grouped K heads
        dict(name="qknb_text_2x77x16x64", op="qknb", batch=2, tokens=77, qheads=16, kheads=4, hd=64,
             a0=16, a1=24, a2=24, dtype="bf16", wdtype="bf16", interleaved=False, merged=True, ptype="i32"),
        # float32 gradients, heads of 96 that turn in part
        dict(name="qknb_f32_2x2047x12x96", op="qknb", batch=2, tokens=2047, qheads=12, kheads=12, hd=96,
             a0=16, a1=24, a2=24, dtype="f32", wdtype="f32", interleaved=True, merged=False, ptype="f32"),
        # scale and shift of the last norm of a small model, one sample: launch latency
        dict(name="lin_last_1x1024x2048", op="lin", rows=1, K=1024, N=2048, dtype="bf16", bias="bf16", silu=True),
        # the six modulation vectors of an image block, a guided pair of samples
        dict(name="lin_image_2x4096x24576", op="lin", rows=2, K=4096, N=24576, dtype="bf16", bias="bf16", silu=True),
        # the six of a video block in float32, one sample
        dict(name="lin_video_1x5120x30720", op="lin", rows=1, K=5120, N=30720, dtype="f32", bias="f32", silu=True),
        # a plain product of sixteen rows (a batch of time steps), an odd number of outputs
        dict(name="lin_batch_16x5120x10007", op="lin", rows=16, K=5120, N=10007, dtype="bf16", bias="", silu=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qkn", "qkn", "qknb", "qknb", "lin", "lin", "lin"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "lin":
        rows = rng.choice([1, 1, 2, 2, 3, 4, 8, 16, 16, rng.randint(1, 64)])
        K = 16 * _log(rng, 8, 512)
        if rng.random() < 0.75:  # most hidden sizes are whole multiples of 64
            K = max(64, K // 64 * 64)
        N = _log(rng, 256, min(49152, 150_000_000 // K))
        if rng.random() < 0.7:
            N = max(256, N // 256 * 256)
        return dict(op=op, rows=rows, K=K, N=N, dtype=dtype, bias=rng.choice(["", "f32", dtype]),
                    silu=rng.random() < 0.6)
    hd = rng.choice([64, 64, 128, 128, 128, 256, 80, 96, 72, 100])
    kheads = rng.choice([1, 2, 8, 24, 40])
    qheads = kheads * rng.choice([1, 1, 4])
    batch = rng.choice([1, 1, 2, 5])
    most = (110_000_000 if op == "qknb" else 140_000_000) // (1 if dtype == "bf16" else 2)
    tokens = _log(rng, 1, max(2, min(65536, most // (batch * (qheads + kheads) * hd))))
    part = hd // 4 * 2 if rng.random() < 0.25 else hd  # some models turn only the first part of a head
    a0 = 2 * rng.randint(1, part // 8)
    a1 = 2 * ((part - a0) // 4)
    return dict(op=op, batch=batch, tokens=tokens, qheads=qheads, kheads=kheads, hd=hd, a0=a0, a1=a1,
                a2=part - a0 - a1, dtype=dtype, wdtype="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                interleaved=rng.random() < 0.55, merged=rng.random() < 0.5, ptype=rng.choice(["i32", "f32"]))


# ---------------------------------------------------------------- inputs


def _normal(g, shape, dt, std=1.0, mean=0.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).add_(mean).to(dt)


def _heads(g, B, S, H, hd, dt):
    """Heads as a projection makes them: each of a size of its own, the channels too, 1 % of the
    elements x 20."""
    x = torch.randn((B, S, H, hd), generator=g, device=DEV)
    x = torch.where(torch.rand((B, S, H, hd), generator=g, device=DEV) < 0.01, x * 20.0, x)
    x *= torch.rand((H, 1), generator=g, device=DEV) * 3.0 + 0.1
    return (x * (torch.rand((hd,), generator=g, device=DEV) + 0.5)).to(dt)


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


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _quantise(w, gs):
    """A weight [N, K] in NVFP4, as a checkpoint is made: packed values [N, K/2] and the scales of
    the blocks of 16 in tiles of 128 rows x 4 blocks, as the package's producers write them."""
    N, K = w.shape
    b = w.float().view(N, K // 16, 16)
    s = (b.abs().amax(dim=-1) * gs / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()
    inv = torch.where(sf > 0, gs / sf, torch.zeros_like(sf))
    v = (b * inv[..., None]).view(N, K)
    mag = v.abs()
    code = torch.zeros_like(v, dtype=torch.uint8)
    for i in range(7):
        mid = (E2M1[i] + E2M1[i + 1]) / 2
        code += (mag >= mid) if i % 2 else (mag > mid)
    code |= (v < 0).to(torch.uint8) << 3
    w4 = code[:, 0::2] | (code[:, 1::2] << 4)
    rows, blocks = -(-N // 128) * 128, -(-(K // 16) // 4) * 4
    tiles = torch.zeros((rows, blocks), dtype=torch.uint8, device=w.device)
    tiles[:N, :K // 16] = s.view(torch.uint8)
    tiles = tiles.view(rows // 128, 4, 32, blocks // 4, 4).permute(0, 3, 2, 1, 4)
    return w4.contiguous(), tiles.reshape(rows, blocks).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case)
    dt = DT[case["dtype"]]
    if case["op"] == "lin":
        rows, K, N = case["rows"], case["K"], case["N"]
        s["x"] = _normal(g, (rows, K), dt, 1.5)
        w = torch.randn((N, K), generator=g, device=DEV).mul_(0.02)
        w *= torch.rand((1, K), generator=g, device=DEV) + 0.5
        w = w.bfloat16()
        s["gs"] = (448.0 * 6.0 / w.abs().amax().float()).reshape(1)
        s["w4"], s["sf"] = _quantise(w, s["gs"])
        s["b"] = _normal(g, (N,), DT[case["bias"]], 0.1) if case["bias"] else None
        return s
    B, S, hq, hk, hd = (case[k] for k in ("batch", "tokens", "qheads", "kheads", "hd"))
    if case["merged"]:  # rows of a merged QKV product, K heads as many as V heads
        qkv = _heads(g, B, S, hq + 2 * hk, hd, dt)
        s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    else:
        s["q"], s["k"] = _heads(g, B, S, hq, hd, dt), _heads(g, B, S, hk, hd, dt)
    s["wq"], s["wk"] = (_normal(g, (hd,), DT[case["wdtype"]], 0.05, 1.0) for _ in range(2))
    if case["op"] == "qknb":  # an attention's gradients, head by head
        s["dq"], s["dk"] = _normal(g, (B, S, hq, hd), dt, 0.01), _normal(g, (B, S, hk, hd), dt, 0.01)
    s["pos"] = _positions(case, g)
    s["axes"] = (case["a0"], case["a1"], case["a2"])
    # the plan a model keeps: the angle per position of every pair, in radians
    s["freqs"] = torch.cat([
        torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=DEV),
                  torch.arange(0, a, 2, dtype=torch.float64, device=DEV) / -a) for a in s["axes"]])
    return s


# ---------------------------------------------------------------- the plain forms


def _turn(f, s, inverse):
    """Heads f [B, S, H, hd] in float32, their pairs turned by the positions' angles."""
    S, axes = f.shape[1], s["axes"]
    n = sum(axes) // 2
    axis_of = [i for i, a in enumerate(axes) for _ in range(a // 2)]
    ang = s["pos"].double().reshape(-1, S, len(axes))[:, :, axis_of] * s["freqs"]  # [1 or B, S, n], 64 bits
    c, sn = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]
    sn = -sn if inverse else sn
    a, b = (f[..., 0:2 * n:2], f[..., 1:2 * n:2]) if s["interleaved"] else (f[..., :n], f[..., n:2 * n])
    o0, o1 = a * c - b * sn, a * sn + b * c
    o = torch.stack([o0, o1], dim=-1).flatten(-2) if s["interleaved"] else torch.cat([o0, o1], dim=-1)
    return torch.cat([o, f[..., 2 * n:]], dim=-1)


def _unit(x):
    """x / rms(x) of each head, and the factor."""
    f = x.float()
    rstd = 1.0 / torch.sqrt(f.square().mean(dim=-1, keepdim=True) + EPS)
    return f * rstd, rstd


def _plain_head_grads(dout, x, w, s):
    g = _turn(dout.float(), s, True)
    xh, rstd = _unit(x)
    gy = g * w.float()
    dx = rstd * (gy - xh * (gy * xh).mean(dim=-1, keepdim=True))
    return dx.to(x.dtype), (g * xh).sum(dim=(0, 1, 2), dtype=torch.float64).to(w.dtype)


def _plain_weight(s):
    """The weight's values times the blocks' scales, [N, K] float32."""
    N, K = s["N"], s["K"]
    w4, sf = s["w4"], s["sf"]
    table = torch.tensor(E2M1 + [-v for v in E2M1], device=DEV)
    codes = torch.stack([w4 & 15, w4 >> 4], dim=-1).view(N, K // 16, 16)
    rows, blocks = sf.shape
    scale = sf.view(rows // 128, blocks // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rows, blocks)
    scale = scale.contiguous().view(torch.float8_e4m3fn)[:N, :K // 16].float()
    return (table[codes.int()] * scale[..., None]).view(N, K)


def _run_plain(s):
    if s["op"] == "qkn":
        return tuple(_turn(_unit(s[k])[0] * s["w" + k].float(), s, False).to(s[k].dtype) for k in ("q", "k"))
    if s["op"] == "qknb":
        (dq, dwq), (dk, dwk) = (_plain_head_grads(s["d" + k], s[k], s["w" + k], s) for k in ("q", "k"))
        return dq, dk, dwq, dwk
    x = s["x"].float()
    a = x / (1.0 + torch.exp(-x)) if s["silu"] else x
    out = (a @ _plain_weight(s).t()) / s["gs"]
    if s["b"] is not None:
        out = out + s["b"].float()
    return out.to(s["x"].dtype)


# ---------------------------------------------------------------- one pass


def _run_own(s):
    m = _lib()
    if s["op"] == "qkn":
        return m.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freqs"], s["axes"],
                              interleaved=s["interleaved"], eps=EPS)
    if s["op"] == "qknb":
        return m.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freqs"],
                                       s["axes"], interleaved=s["interleaved"], eps=EPS)
    return m.linear_nvfp4(s["x"], s["w4"], s["sf"], s["gs"], bias=s["b"], silu=s["silu"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- binary64


def _exact_heads(x, w, s, lo, hi):
    """The definition on tokens lo..hi, each pair a complex number times e^(i * angle)."""
    n = sum(s["axes"]) // 2
    pos = s["pos"].double().reshape(-1, s["tokens"], 3)[:, lo:hi]
    turn = torch.empty((pos.shape[0], hi - lo, n), dtype=torch.complex128, device=DEV)
    first = 0
    for i, a in enumerate(s["axes"]):
        for j in range(a // 2):
            ang = pos[:, :, i] * 10000.0 ** (-2.0 * j / a)
            turn[:, :, first + j] = torch.complex(torch.cos(ang), torch.sin(ang))
        first += a // 2
    d = x * (x.pow(2).sum(dim=-1, keepdim=True) / x.shape[-1] + EPS) ** -0.5 * w
    if s["interleaved"]:
        z = torch.view_as_complex(d[..., :2 * n].reshape(*d.shape[:3], n, 2))
    else:
        z = torch.complex(d[..., :n].contiguous(), d[..., n:2 * n].contiguous())
    z = z * turn[:, :, None]
    turned = torch.view_as_real(z).flatten(-2) if s["interleaved"] else torch.cat([z.real, z.imag], dim=-1)
    return torch.cat([turned, d[..., 2 * n:]], dim=-1)


def _exact_qk(s, name, grads):
    x, w = s[name], s["w" + name]
    B, S, H, hd = x.shape
    outs, dw = [], torch.zeros(hd, dtype=torch.float64, device=DEV)
    block = max(1, (1 << 24) // (B * H * hd))
    for lo in range(0, S, block):
        hi = min(S, lo + block)
        xd = x[:, lo:hi].double().requires_grad_(grads)
        wd = w.double().requires_grad_(grads)
        out = _exact_heads(xd, wd, s, lo, hi)
        if not grads:
            outs.append(out)
            continue
        gx, gw = torch.autograd.grad(out, (xd, wd), s["d" + name][:, lo:hi].double())
        outs.append(gx)
        dw += gw
    return torch.cat(outs, dim=1), dw


def _exact_lin(s):
    """The sum over k in binary64, some output columns at a time; the scale of (n, block) is read from
    its place in the tiles."""
    N, K = s["N"], s["K"]
    a = s["x"].double()
    if s["silu"]:
        a = a * torch.sigmoid(a)
    value = torch.tensor([(-1.0) ** (c >> 3) * ((c & 1) / 2 if (c >> 1) & 3 == 0 else
                                                (1 + (c & 1) / 2) * 2.0 ** (((c >> 1) & 3) - 1)) for c in range(16)],
                         dtype=torch.float64, device=DEV)
    blk = torch.arange(K // 16, device=DEV)
    flat = s["sf"].reshape(-1).view(torch.float8_e4m3fn)
    out = torch.empty((s["rows"], N), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 24) // K)
    for lo in range(0, N, step):
        n = torch.arange(lo, min(N, lo + step), device=DEV)
        byte = s["w4"][n].int()
        w = torch.empty((len(n), K), dtype=torch.float64, device=DEV)
        w[:, 0::2], w[:, 1::2] = value[byte % 16], value[byte // 16]
        r = n[:, None]
        at = ((r // 128) * (s["sf"].shape[1] // 4) + blk // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + blk % 4
        w *= flat[at].double().repeat_interleave(16, dim=1)
        out[:, lo:lo + len(n)] = a @ w.t()
    out /= s["gs"].double()
    return out if s["b"] is None else out + s["b"].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lin":
        return _exact_lin(s)
    (q, dwq), (k, dwk) = (_exact_qk(s, n, case["op"] == "qknb") for n in ("q", "k"))
    return (q, k, dwq, dwk) if case["op"] == "qknb" else (q, k)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "lin":
        rows, K, N = case["rows"], case["K"], case["N"]
        bias = {"": 0, "bf16": 2, "f32": 4}[case["bias"]]
        return {"bytes": N * K // 2 + N * K // 16 + rows * K * e + rows * N * e + N * bias + 4,
                "flops": 2 * rows * N * K}
    tokens = case["batch"] * case["tokens"]
    n = tokens * (case["qheads"] + case["kheads"]) * case["hd"]
    pos_rows = tokens if case["tokens"] == 1 else case["tokens"]
    pairs = (case["a0"] + case["a1"] + case["a2"]) // 2
    we = 4 if case["wdtype"] == "f32" else 2
    small = pos_rows * 12 + pairs * 8 + 2 * case["hd"] * we
    if case["op"] == "qkn":
        return {"bytes": 2 * n * e + small, "flops": 7 * n}
    return {"bytes": 3 * n * e + small + 2 * case["hd"] * we, "flops": 15 * n}
