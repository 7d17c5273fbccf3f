"""Norms that a model is trained through: what they compute, on which sizes, and what they cannot do without.

* ln_save: LayerNorm + modulate of rows [B, T, D], rounded once, with what its gradient needs: the rows' mean and
  1/std, and the rows themselves as a checkpoint in 8 bits.
* ln_back: its gradients, from the checkpoint or from the rows; the residual stream's gradient may be added.
* gn: group norm over the positions of channels-last images [N, C, H, W], with scale and shift per image, SiLU, and
  again what the gradient needs.
* gn_back: its gradients.

A checkpoint holds E4M3 codes and, for each 32 neighbouring channels, the least power of two (as its E8M0 code) at
which none of them exceeds 448.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _ln(name, op, B, T, D, ckpt, **more):
    return dict(name=name, op=op, B=B, T=T, D=D, ckpt=ckpt, **more)


def _gn(name, op, N, H, W, C, G, type="bf16", params="same", act="silu", mod=False, **more):
    return dict(name=name, op=op, N=N, H=H, W=W, C=C, G=G, type=type, params=params, act=act, mod=mod, **more)


def listed():
    return [
        # a short text stream's norm in a training step: latency
        _ln("ln_save_text", "ln_save", 1, 128, 2048, True),
        # the image tokens of one training sample
        _ln("ln_save_image", "ln_save", 1, 4216, 4096, True),
        # the gradient of a pair of samples whose rows were kept as they are, added to the residual stream's
        _ln("ln_back_pair", "ln_back", 2, 1140, 4096, False, res=True),
        # the gradient of the image tokens from their checkpoint
        _ln("ln_back_image", "ln_back", 1, 4216, 4096, True, res=False),
        # a batch of a small model, an odd width and length
        _ln("ln_back_batch", "ln_back", 8, 4173, 1160, True, res=True),
        # the lowest level of a denoiser, one image: latency
        _gn("gn_bottom", "gn", 1, 8, 8, 1280, 32, mod=True, save=False, ckpt=False),
        # the first level of an image decoder
        _gn("gn_decode", "gn", 1, 128, 128, 512, 32, save=False, ckpt=False),
        # its last one, at the image's full size
        _gn("gn_decode_full", "gn", 1, 1024, 1024, 128, 32, save=False, ckpt=False),
        # odd images in 32 bits, ten channels a group, no activation
        _gn("gn_odd", "gn", 3, 93, 61, 320, 32, type="fp32", act="none", save=True, ckpt=False),
        # a training step's norm in a denoiser, the input kept in 8 bits
        _gn("gn_save", "gn", 8, 64, 64, 640, 32, type="fp16", params="fp32", mod=True, save=True, ckpt=True),
        # the gradient of a denoiser's norm, ten channels a group, from checkpoints
        _gn("gn_back_batch", "gn_back", 16, 64, 64, 320, 32, mod=True, ckpt=True),
        # the gradient in a decoder's training, one large image
        _gn("gn_back_decode", "gn_back", 1, 512, 512, 256, 32, params="fp32", ckpt=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        op = rng.choice(["ln_save", "ln_back", "ln_back"])
        B, D = rng.choice([1, 1, 2, 3, 8, 16]), 8 * _log(rng, 1, 1024)
        c = dict(op=op, B=B, T=_log(rng, 1, min(65536, 38_000_000 // (B * D))), D=D, ckpt=rng.random() < 0.7)
        if op == "ln_back":
            c["res"] = rng.random() < 0.5
        return c
    op = rng.choice(["gn", "gn", "gn_back"])
    per = rng.choice([1, 2, 4, 5, 8, 10, 12, 16, 20, 30, 40])  # channels a group
    G = rng.choice([g for g in (1, 8, 16, 32, 48) if g * per % 8 == 0])
    C, type = G * per, rng.choice(["bf16", "bf16", "fp16", "fp32"])
    most = 60_000_000 // (2 if type == "fp32" else 1) // C
    N = rng.choice([1, 1, 2, 3, 8, 16])
    H = _log(rng, 4, math.isqrt(min(1024 * 1024, most // N)))
    W = min(_log(rng, max(4, H // 2), 2 * H + 3), most // (N * H))
    save = op == "gn_back" or rng.random() < 0.5
    c = dict(op=op, N=N, H=H, W=W, C=C, G=G, type=type, params=rng.choice(["same", "fp32"]),
             act=rng.choice(["silu", "silu", "none"]), mod=rng.random() < 0.4,
             ckpt=save and C % 32 == 0 and rng.random() < 0.5)
    if op == "gn":
        c["save"] = save
    return c


def work(case):
    c = case
    if c["op"] in ("ln_save", "ln_back"):
        rows, D = c["B"] * c["T"], c["D"]
        kept = D + -(-D // 32)
        vec = c["B"] * D * 2
        if c["op"] == "ln_save":
            return {"bytes": rows * (4 * D + 8 + (kept if c["ckpt"] else 0)) + 2 * vec, "flops": rows * D * 8}
        row = 2 * D + (kept if c["ckpt"] else 2 * D) + 8 + 2 * D + (2 * D if c["res"] else 0)
        return {"bytes": rows * row + 3 * vec, "flops": rows * D * 14}
    es, n, N, C = DTYPES[c["type"]].itemsize, c["N"] * c["H"] * c["W"] * c["C"], c["N"], c["C"]
    ws = 4 if c["params"] == "fp32" else es
    stats, kept = N * c["G"] * 8, n + n // 32
    mod = 2 * N * C * es if c["mod"] else 0
    if c["op"] == "gn":
        return {"bytes": 2 * n * es + 2 * C * ws + mod + (stats if c["save"] else 0) + (kept if c["ckpt"] else 0),
                "flops": n * (12 if c["act"] == "silu" else 7)}
    return {"bytes": 2 * n * es + (kept if c["ckpt"] else n * es) + stats + 4 * C * ws + 2 * mod,
            "flops": n * (24 if c["act"] == "silu" else 14)}


# ----------------------------------------------------------------- inputs

def _normal(shape, g, std=1.0, mean=0.0, dtype=torch.bfloat16):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=g)
    return x.to(dtype)


def _activations(rows, C, g, dtype):
    """Rows whose channels have levels and spreads of their own, one channel in a hundred a large one."""
    x = torch.empty((rows, C), dtype=torch.float32, device="cuda").normal_(generator=g)
    spread = torch.exp(0.3 * torch.empty(C, device="cuda").normal_(generator=g))
    spread = torch.where(torch.rand(C, device="cuda", generator=g) < 0.01, 20 * spread, spread)
    return x.mul_(spread).add_(0.5 * torch.empty(C, device="cuda").normal_(generator=g)).to(dtype)


def _checkpoint(x):
    """(E4M3 codes, E8M0 codes) of x [..., C] in blocks of 32 channels, as bytes; exact up to the codes' rounding."""
    C, tail = x.shape[-1], -x.shape[-1] % 32
    blocks = torch.nn.functional.pad(x.float(), (0, tail)).unflatten(-1, (-1, 32))
    top = blocks.abs().amax(-1)
    m, e = torch.frexp(top)  # m in [0.5, 1): 448 is 0.875 * 2^9
    e = torch.where(top > 0, e - 9 + (m > 0.875), -126).clamp(min=-126)
    power = ((127 - e) << 23).to(torch.int32).view(torch.float32)  # 2^-e
    codes = (blocks * power[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.flatten(-2)[..., :C].contiguous(), (e + 127).to(torch.uint8)


def _kept(codes, scales):
    """The values that a checkpoint stands for, in 32 bits."""
    C = codes.shape[-1]
    v = codes.view(torch.float8_e4m3fn).float()
    s = scales.view(torch.float8_e8m0fnu).float()
    return v * s.repeat_interleave(32, -1)[..., :C]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] in ("ln_save", "ln_back"):
        B, T, D = c["B"], c["T"], c["D"]
        x = _activations(B * T, D, g, torch.bfloat16).view(B, T, D)
        # scale and shift are slices of one embedding, their gradients' places too
        emb = _normal((B, 6 * D), g, 0.2)
        s = dict(c=c, scale=emb[:, :D], shift=emb[:, D:2 * D])
        if c["op"] == "ln_save":
            return dict(s, x=x)
        y = x.double()
        mean = y.mean(-1)
        stats = torch.stack([mean, (y.var(-1, correction=0) + EPS).rsqrt()], -1).float()
        del y
        s.update(x=None if c["ckpt"] else x, saved=(stats, *(_checkpoint(x) if c["ckpt"] else (None, None))),
                 dy=_normal((B, T, D), g, 0.1), dres=_normal((B, T, D), g, 0.1) if c["res"] else None)
        return s
    N, H, W, C, G, dtype = c["N"], c["H"], c["W"], c["C"], c["G"], DTYPES[c["type"]]
    wtype = torch.float32 if c["params"] == "fp32" else dtype
    x = _activations(N * H * W, C, g, dtype)

    def image(t):
        return t.view(N, H, W, C).permute(0, 3, 1, 2)

    s = dict(c=c, weight=_normal((C,), g, 0.2, 1.0, wtype), bias=_normal((C,), g, 0.2, 0.0, wtype),
             act=None if c["act"] == "none" else c["act"], scale=None, shift=None)
    if c["mod"]:
        emb = _normal((N, 2 * C), g, 0.2, 0.0, dtype)
        s.update(scale=emb[:, :C], shift=emb[:, C:])
    if c["op"] == "gn":
        return dict(s, x=image(x))
    y = x.view(N, H * W, G, C // G).double()
    mean = y.mean((1, 3))
    var = (y - mean[:, None, :, None]).square_().mean((1, 3))
    del y
    stats = torch.stack([mean, (var + EPS).rsqrt()], -1).float()
    codes, scales = None, None
    if c["ckpt"]:
        codes, scales = (image(t) if t.shape[1] == C else t.view(N, H, W, -1).permute(0, 3, 1, 2)
                         for t in _checkpoint(x))
    s.update(x=None if c["ckpt"] else image(x), saved=(stats, codes, scales),
             dy=image(_normal((N * H * W, C), g, 0.1, 0.0, dtype)))
    return s


# -------------------------------------------------------------------- run

def run(state):
    s = state
    c = s["c"]
    if own:
        from dit_adaln_norm_gb300 import ops
        if c["op"] == "ln_save":
            y, saved = ops.ln_modulate_save(s["x"], s["scale"], s["shift"], EPS, checkpoint=c["ckpt"])
            return y, *_as_values(saved)
        if c["op"] == "ln_back":
            return ops.ln_modulate_backward(s["dy"], s["x"], s["scale"], s["saved"], dres=s["dres"])
        if c["op"] == "gn" and c["save"]:
            y, saved = ops.group_norm_save(s["x"], c["G"], s["weight"], s["bias"], EPS, act=s["act"], scale=s["scale"],
                                           shift=s["shift"], checkpoint=c["ckpt"])
            return y, *_as_values(saved)
        if c["op"] == "gn":
            return ops.group_norm(s["x"], c["G"], s["weight"], s["bias"], EPS, act=s["act"], scale=s["scale"],
                                  shift=s["shift"])
        return ops.group_norm_backward(s["dy"], s["x"], c["G"], s["weight"], s["bias"], s["saved"], act=s["act"],
                                       scale=s["scale"], shift=s["shift"])
    return {"ln_save": _plain_ln, "ln_back": _plain_ln_back, "gn": _plain_gn, "gn_back": _plain_gn_back}[c["op"]](s, c)


def _as_values(saved):
    stats, codes, scales = saved
    if codes is None:
        return stats, None, None
    return stats, codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _plain_ln(s, c):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    rstd = (d.square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = (d * rstd * (1 + s["scale"].float()[:, None]) + s["shift"].float()[:, None]).bfloat16()
    kept = _checkpoint(s["x"]) if c["ckpt"] else (None, None)
    return y, *_as_values((torch.cat([mean, rstd], -1), *kept))


def _plain_ln_back(s, c):
    stats, codes, scales = s["saved"]
    x = _kept(codes, scales) if c["ckpt"] else s["x"].float()
    mean, rstd = stats[..., :1], stats[..., 1:]
    n = (x - mean) * rstd
    dy = s["dy"].float()
    g = dy * (1 + s["scale"].float()[:, None])
    dx = rstd * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    if c["res"]:
        dx = dx + s["dres"].float()
    return dx.bfloat16(), (dy * n).sum(1).bfloat16(), dy.sum(1).bfloat16()


def _rows(t):
    """[N, C, H, W] in channels-last memory as [N, H*W, C]."""
    return t.permute(0, 2, 3, 1).flatten(1, 2)


def _image(t, c):
    return t.view(c["N"], c["H"], c["W"], -1).permute(0, 3, 1, 2)


def _gains(s, c):
    """z = n * a + b: the gain and offset [N or 1, 1, C] of the normalised values."""
    w, b = s["weight"].float()[None, None], s["bias"].float()[None, None]
    if not c["mod"]:
        return w, b
    o = 1 + s["scale"].float()[:, None]
    return w * o, b * o + s["shift"].float()[:, None]


def _plain_gn(s, c):
    x = _rows(s["x"]).float().unflatten(2, (c["G"], -1))
    mean = x.mean((1, 3), keepdim=True)
    d = x - mean
    rstd = (d.square().mean((1, 3), keepdim=True) + EPS).rsqrt()
    a, b = _gains(s, c)
    z = (d * rstd).flatten(2) * a + b
    if c["act"] == "silu":
        z = z / (1 + (-z).exp())
    y = _image(z.to(s["x"].dtype), c)
    if not c["save"]:
        return y
    kept = [_image(t, c) for t in _checkpoint(_rows(s["x"]))] if c["ckpt"] else (None, None)
    return y, *_as_values((torch.stack([mean.flatten(1), rstd.flatten(1)], -1), *kept))


def _plain_gn_back(s, c):
    stats, codes, scales = s["saved"]
    x = _kept(_rows(codes).contiguous(), _rows(scales).contiguous()) if c["ckpt"] else _rows(s["x"]).float()
    mean, rstd = (stats[:, None, :, i].repeat_interleave(c["C"] // c["G"], 2) for i in range(2))
    n = (x - mean) * rstd
    a, b = _gains(s, c)
    dz = _rows(s["dy"]).float()
    if c["act"] == "silu":
        z = n * a + b
        p = 1 / (1 + (-z).exp())
        dz = dz * (p * (1 + z * (1 - p)))
    g = dz * a
    m1, m2 = (t.unflatten(2, (c["G"], -1)).mean((1, 3)).repeat_interleave(c["C"] // c["G"], 1)[:, None] for t in (g, g * n))
    dx = _image((rstd * (g - m1 - n * m2)).to(s["dy"].dtype), c)
    s0, s1 = dz.sum(1), (dz * n).sum(1)  # [N, C]
    if not c["mod"]:
        return dx, s1.sum(0).to(s["weight"].dtype), s0.sum(0).to(s["bias"].dtype), None, None
    o = 1 + s["scale"].float()
    w, b = s["weight"].float(), s["bias"].float()
    return (dx, (o * s1).sum(0).to(s["weight"].dtype), (o * s0).sum(0).to(s["bias"].dtype),
            (w * s1 + b * s0).to(s["scale"].dtype), s0.to(s["shift"].dtype))


# ------------------------------------------------------------------ exact

def _power(k):
    """2^k in 64 bits, from its bits: the library's powers of two are not all exact."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_checkpoint(x):
    """The codes' and scales' values of x [rows, C] in 64 bits, from the format's definition."""
    rows, C = x.shape
    codes, scales = torch.empty_like(x), torch.empty((rows, -(-C // 32)), dtype=torch.float64, device=x.device)
    for b in range(-(-C // 32)):
        v = x[:, 32 * b:32 * b + 32]
        top = v.abs().amax(1)
        k = torch.ceil(torch.log2(top / 448)).clamp(min=-126)  # exact but for a step at the powers' borders
        k = torch.where(top > 448 * _power(k), k + 1, k)
        k = torch.where((top <= 448 * _power(k - 1)) & (k > -126), k - 1, k)
        scales[:, b] = _power(k)
        u = v / scales[:, b:b + 1]
        # E4M3: three bits behind the leading one, steps of 2^-9 at least; torch rounds ties to even
        step = _power((torch.frexp(u).exponent - 1).clamp(min=-6) - 3)
        codes[:, 32 * b:32 * b + 32] = torch.round(u / step) * step
    return codes, scales


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "ln_save":
        x = s["x"].double()
        o, sh = 1 + s["scale"].double(), s["shift"].double()
        mean = x.sum(2) / c["D"]
        var = ((x - mean[..., None]) ** 2).sum(2) / c["D"]
        rstd = 1 / torch.sqrt(var + EPS)
        y = torch.addcmul(sh[:, None], (x - mean[..., None]) * rstd[..., None], o[:, None])
        if not c["ckpt"]:
            return y, torch.stack([mean, rstd], 2), None, None
        q, k = _exact_checkpoint(x.flatten(0, 1))
        return y, torch.stack([mean, rstd], 2), q.view(x.shape), k.view(c["B"], c["T"], -1)
    if c["op"] == "ln_back":
        stats, codes, scales = s["saved"]
        dx = torch.empty(s["dy"].shape, dtype=torch.float64, device="cuda")
        do, dsh = (torch.empty((c["B"], c["D"]), dtype=torch.float64, device="cuda") for _ in range(2))
        for b in range(c["B"]):
            x = _exact_kept(codes[b], scales[b]) if c["ckpt"] else s["x"][b].double()
            mean, r = stats[b].double().unbind(1)
            n = (x - mean[:, None]) * r[:, None]
            dy = s["dy"][b].double()
            do[b], dsh[b] = torch.einsum("td,td->d", dy, n), dy.sum(0)
            g = dy * (1 + s["scale"][b].double())
            dx[b] = r[:, None] * (g - g.sum(1, keepdim=True) / c["D"] - n * (torch.einsum("td,td->t", g, n) / c["D"])[:, None])
            if c["res"]:
                dx[b] += s["dres"][b]
        return dx, do, dsh
    N, H, W, C, G = c["N"], c["H"], c["W"], c["C"], c["G"]
    per, count = C // G, H * W * (C // G)
    w, b = s["weight"].double(), s["bias"].double()
    y = torch.empty((N, H * W, C), dtype=torch.float64, device="cuda")
    stats = torch.empty((N, G, 2), dtype=torch.float64, device="cuda")
    dw, db, do, dsh = (torch.zeros(k, dtype=torch.float64, device="cuda") for k in ((C,), (C,), (N, C), (N, C)))
    codes = scales = None
    if c["op"] == "gn" and c["ckpt"]:
        codes, scales = (torch.empty((N, H * W, k), dtype=torch.float64, device="cuda") for k in (C, C // 32))
    for i in range(N):
        if c["op"] == "gn":
            x = s["x"][i].reshape(C, H * W).double()
            if c["ckpt"]:
                codes[i], scales[i] = _exact_checkpoint(x.T.contiguous())
        elif c["ckpt"]:
            x = _exact_kept(s["saved"][1][i].reshape(C, -1).T, s["saved"][2][i].reshape(C // 32, -1).T).T
        else:
            x = s["x"][i].reshape(C, H * W).double()
        for h in range(G):
            at = slice(h * per, (h + 1) * per)
            if c["op"] == "gn":
                mean = x[at].sum() / count
                r = 1 / torch.sqrt(((x[at] - mean) ** 2).sum() / count + EPS)
                stats[i, h, 0], stats[i, h, 1] = mean, r
            else:
                mean, r = s["saved"][0][i, h].double()
            n = (x[at] - mean) * r
            o = 1 + s["scale"][i, at].double() if c["mod"] else torch.ones(per, dtype=torch.float64, device="cuda")
            z = (n * w[at, None] + b[at, None]) * o[:, None]
            if c["mod"]:
                z += s["shift"][i, at].double()[:, None]
            p = torch.sigmoid(z) if c["act"] == "silu" else None
            if c["op"] == "gn":
                y[i, :, at] = (z if p is None else z * p).T
                continue
            dz = s["dy"][i, at].reshape(per, -1).double()
            if p is not None:
                dz = dz * (p + z * p * (1 - p))
            t0, t1 = dz.sum(1), (dz * n).sum(1)
            dsh[i, at], do[i, at] = t0, w[at] * t1 + b[at] * t0
            dw[at] += o * t1
            db[at] += o * t0
            g = dz * (w[at] * o)[:, None]
            y[i, :, at] = (r * (g - g.sum() / count - n * ((g * n).sum() / count))).T
    y = _image(y, c)
    if c["op"] == "gn_back":
        return y, dw, db, *((do, dsh) if c["mod"] else (None, None))
    if not c["save"]:
        return y
    return y, stats, *((_image(codes, c), _image(scales, c)) if c["ckpt"] else (None, None))


def _exact_kept(codes, scales):
    """The values of a checkpoint's rows, decoded from the codes' bits in 64 bits."""
    u = codes.to(torch.int64)
    e, m = (u >> 3) & 15, (u & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _power(e - 10))
    v = torch.where(u >= 128, -v, v)
    k = _power(scales.to(torch.int64) - 127)
    return v * k.repeat_interleave(32, 1)[:, :v.shape[1]]
