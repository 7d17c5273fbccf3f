"""64-bit references and error bounds for the training operators' tests.

Bounds count roundings: HALF[t] is half a step of a type relative to the value, and E a bound on
what a chain of fp32 operations adds (some 128 roundings of half a step of fp32 each: a thread's
sums are of a few dozen terms, then trees)."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-37, torch.float16: 2.0 ** -25, torch.float32: 1e-37}  # half the least step
E = 128 * 2.0 ** -24


def power(k):
    """2^k as fp64, from its bits (k a tensor of whole numbers)."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def checkpoint(x):
    """(codes, scales) as the format defines them: x [..., C] of any type, bytes out."""
    C = x.shape[-1]
    v = torch.nn.functional.pad(x.double(), (0, -C % 32)).unflatten(-1, (-1, 32))
    top = torch.where(v.isnan(), 0.0, v.abs()).amax(-1)
    m, e = torch.frexp(top)
    k = torch.where(top > 0, e - 9 + (m > 0.875), -126).clamp(min=-126)
    k = torch.where(top.isinf(), 120, k)
    u = v * power(-k)[..., None]
    codes = u.clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.flatten(-2)[..., :C], (k + 127).to(torch.uint8)


def restore(codes, scales):
    """The values of a checkpoint [..., C], in fp64."""
    C = codes.shape[-1]
    v = codes.contiguous().view(torch.float8_e4m3fn).double()
    return v * power(scales.to(torch.int64) - 127).repeat_interleave(32, -1)[..., :C]


def bound(want, dtype, extra):
    """Whether a result of `dtype` may be this far from the 64-bit value."""
    return want.abs() * HALF[dtype] + extra * (1 + HALF[dtype]) + TINY[dtype]


def assert_near(got, want, extra, what=""):
    got, lim = got.double(), bound(want, got.dtype, extra)
    bad = ~((got - want).abs() <= lim)
    bad &= ~(got.isnan() & want.isnan())
    if bool(bad.any()):
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {at}: {float(got[at])} "
                             f"for {float(want[at])}, bound {float(lim.expand_as(want)[at])}")


# ------------------------------------------------------------------- LayerNorm

def ln_forward(x, scale, shift, eps):
    """y, stats and how far fp32 may take each from them."""
    x, o, sh = x.double(), 1 + scale.double()[:, None], shift.double()[:, None]
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    n = (x - mean) * rstd
    top = x.abs().amax(-1, keepdim=True)
    y = n * o + sh
    # the mean is off by E of the largest value, 1/std by E of it and by what the
    # differences x - mean lose
    far = E * (1 + top * rstd)
    return y, torch.cat([mean, rstd], -1), far * (1 + n.abs()) * o.abs() + E * sh.abs(), \
        torch.cat([E * top, far * rstd], -1)


def ln_backward(dy, x, stats, scale, dres, rows_per_thread):
    """(dx, dscale, dshift) and their fp32 errors; x in fp64."""
    mean, rstd = stats.double()[..., :1], stats.double()[..., 1:]
    o, dy = 1 + scale.double()[:, None], dy.double()
    n = (x - mean) * rstd
    g = dy * o
    avg = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    dx = rstd * (g - avg(g) - n * avg(g * n))
    ex = E * rstd * (g.abs() + avg(g.abs()) + n.abs() * avg((g * n).abs()))
    if dres is not None:
        dx = dx + dres.double()
        ex = ex + E * dres.double().abs()
    many = (rows_per_thread + 64) * 2.0 ** -24
    return (dx, (dy * n).sum(1), dy.sum(1)), (ex, many * (dy * n).abs().sum(1), many * dy.abs().sum(1))


# ------------------------------------------------------------------ group norm

def rows(t):
    """An image tensor as [N, S, C]."""
    return t if t.dim() == 3 else t.movedim(1, -1).flatten(1, -2)


def gains(weight, bias, scale, shift, N, C, device):
    one = torch.ones((1, C), dtype=torch.float64, device=device)
    w = one if weight is None else weight.double()[None]
    b = 0 * one if bias is None else bias.double()[None]
    o = one.expand(N, C) if scale is None else 1 + scale.double()
    t = (0 * one).expand(N, C) if shift is None else shift.double()
    return w, b, o, t


def gn_forward(x, groups, weight, bias, eps, act, scale, shift):
    """y, stats [N, groups, 2] and their fp32 errors."""
    x = rows(x).double()
    N, S, C = x.shape
    v = x.unflatten(2, (groups, -1))
    mean = v.mean((1, 3), keepdim=True)
    rstd = ((v - mean).square().mean((1, 3), keepdim=True) + eps).rsqrt()
    n = ((v - mean) * rstd).flatten(2)
    w, b, o, t = gains(weight, bias, scale, shift, N, C, x.device)
    a, c = (w * o)[:, None], (b * o + t)[:, None]
    z = n * a + c
    top = v.abs().amax((1, 3), keepdim=True)
    far = E * (1 + top * rstd)
    ez = far.expand_as(v).flatten(2) * (1 + n.abs()) * a.abs() + E * (b * o).abs()[:, None] + E * t.abs()[:, None]
    y = z
    if act:
        p = torch.sigmoid(z)
        y = z * p
        # the derivative is at most 1.1; exp is within 2 + 1.2|z| steps, the quotient within 3
        ez = 1.1 * ez + y.abs() * (8 + 1.2 * z.abs()) * 2.0 ** -23 + 1e-30
    return y, torch.cat([mean, rstd], -1)[:, 0], ez, \
        torch.cat([E * top, far * rstd], -1)[:, 0]


def gn_backward(dy, x, groups, weight, bias, stats, act, scale, shift):
    """[dx, dweight, dbias, dscale, dshift] and their fp32 errors; x [N, S, C] in fp64."""
    dy = rows(dy).double()
    N, S, C = x.shape
    per = C // groups
    mean, rstd = (stats.double()[:, None, :, i].repeat_interleave(per, 2) for i in range(2))
    w, b, o, t = gains(weight, bias, scale, shift, N, C, x.device)
    a, c = (w * o)[:, None], (b * o + t)[:, None]
    n = (x - mean) * rstd
    dz, ez = dy, 4 * 2.0 ** -24 * dy.abs()
    if act:
        z = n * a + c
        p = torch.sigmoid(z)
        dz = dy * (p * (1 + z * (1 - p)))
        # z is off by some steps of its terms, the second derivative at most 1/2; the
        # function units' error on p counts p and z * p, and again in 1 - p
        off = 8 * 2.0 ** -24 * ((n * a).abs() + (b * o).abs()[:, None] + t.abs()[:, None])
        ez = dy.abs() * (0.5 * off + (p + z.abs() * p) * (16 + 2.4 * z.abs()) * 2.0 ** -23)
    g = dz * a
    avg = lambda v: v.unflatten(2, (groups, -1)).mean((1, 3)).repeat_interleave(per, 1)[:, None]  # noqa: E731
    dx = rstd * (g - avg(g) - n * avg(g * n))
    eg = ez * a.abs() + E * g.abs()
    ex = rstd * (eg + avg(eg) + n.abs() * avg(eg * n.abs()))
    s0, s1 = dz.sum(1), (dz * n).sum(1)
    e0, e1 = (ez + E * dz.abs()).sum(1), ((ez + E * dz.abs()) * n.abs()).sum(1)
    grads = [dx, (o * s1).sum(0), (o * s0).sum(0), w * s1 + b * s0, s0]
    errs = [ex, (o.abs() * e1).sum(0) * 2, (o.abs() * e0).sum(0) * 2, 2 * (w.abs() * e1 + b.abs() * e0), e0]
    if weight is None:
        grads[1] = grads[2] = None
    if scale is None:
        grads[3] = grads[4] = None
    return grads, errs
