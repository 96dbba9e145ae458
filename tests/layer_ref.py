"""64-bit references of the layer operators (residual norm, 4-bit linear,
gated pair) and error bounds for their fp32 kernels.  CPU, numpy and torch
float64; shares no code with the package.
"""
import numpy as np
import torch

U32 = 2.0 ** -24          # half a step of fp32, relative
HALF = {torch.float32: U32, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


class Matrix:
    """A seeded 4-bit matrix: codes, fp16 scale and bias, and its 64-bit values."""

    def __init__(self, n, k, group, seed=0, centred=True):
        g = torch.Generator().manual_seed(seed * 1000003 + n * 31 + k * 7 + group)
        self.n, self.k, self.group = n, k, group
        self.q = torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8)
        self.s = (torch.rand(n, k // group, generator=g) * 0.015 + 0.005).half()
        self.b = (torch.randn(n, k // group, generator=g) * 0.01 - (7.5 * self.s.float() if centred else 0)).half()

    def values(self):
        s, b = (v.double().repeat_interleave(self.group, 1) for v in (self.s, self.b))
        return s * self.q.double() + b

    def product(self, x):
        """(x W^T, bound on the kernel's fp32 error) for float64 rows x.

        Bound: a group's two sums are at most 64 additions in the matrix
        core, each off by at most 2^-23 of the sum of magnitudes; then two
        fused multiply-adds a group and up to 16 partial sums in fp32."""
        y = x @ self.values().t()
        s, b = (v.double().abs().repeat_interleave(self.group, 1) for v in (self.s, self.b))
        mag = x.abs() @ (s * self.q.double() + b).t()
        groups = self.k // self.group
        return y, (2 * 64 + 2 * groups + 16) * U32 * mag


def e4m3_product_error(m, x):
    """Bound on what the e4m3 matrix core adds to the error: it aligns the 64
    products of an instruction to the largest one and keeps 13 bits of that at
    the least (the outputs that take this path have 8 bits), so each of the 64
    is off by at most 2^-13 of the largest; likewise the group sum of x, which
    the bias multiplies."""
    t, k = x.shape
    s, b = m.s.double().abs(), m.b.double().abs()
    top = x.abs().view(t, k // m.group, m.group).amax(2)            # the largest product is at most 15 of these
    return 64 * 2.0 ** -13 * (top @ (15 * s + b).t())


def e4m3_rows(v, kind):
    """float32 rows -> (codes float8_e4m3fn, scale, float64 values); any scales
    will do for inputs, these use the whole range of codes."""
    t, k = v.shape
    if kind == "none":
        c = v.clamp(-448, 448).to(torch.float8_e4m3fn)
        return c, None, c.double()
    if kind == "row":
        s = (v.abs().amax(1) / 448).clamp_min(2.0 ** -126).float()
        c = (v / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        return c, s, c.double() * s.double()[:, None]
    amax = v.abs().view(t, k // 32, 32).amax(2).double().numpy()
    e = block_exponent(amax)
    s = torch.from_numpy(np.exp2(e.astype(np.float64)))
    c = (v.double().view(t, k // 32, 32) / s[..., None]).clamp(-448, 448).float().to(torch.float8_e4m3fn).view(t, k)
    values = (c.double().view(t, k // 32, 32) * s[..., None]).view(t, k)
    return c, torch.from_numpy((e + 127).astype(np.uint8)), values


def block_exponent(amax):
    """Smallest E >= -127 with amax <= 448 * 2^E."""
    with np.errstate(divide="ignore"):
        m, e = np.frexp(np.asarray(amax, dtype=np.float64) / 448.0)
    e = np.where(m == 0.5, e - 1, e)
    return np.where(np.asarray(amax) == 0, -127, np.clip(e, -127, 127)).astype(np.int64)


def check_rounded(got, ref, err, dtype, what):
    """got (a tensor of dtype) against ref within err and half a step of dtype."""
    g = got.double().cpu()
    tol = err + HALF[dtype] * (ref.abs() + err) + 2.0 ** -140
    bad = ~((g - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((g - ref).abs().max()), float(tol.max()))


def scale_values(scale):
    """Scales as float64: fp32 a row [t, 1], or bytes [t, width/32]."""
    s = scale.cpu()
    if s.dtype == torch.float32:
        return s.double()[:, None]
    return torch.exp2(s.view(torch.uint8).double() - 127)


def check_codes(codes, scale, ref, err, what):
    """8-bit rows against float64 values ref known to +-err: the scale is the
    defined one for some value within err, and every code is the nearest."""
    s = scale_values(scale)
    t, w = ref.shape
    n = s.shape[1]
    blocks = ref.abs().view(t, n, w // n)
    eb = err.view(t, n, w // n)
    hi, lo = (blocks + eb).amax(2), (blocks - eb).clamp_min(0).amax(2)
    if scale.dtype == torch.float32:
        assert bool(((s <= (hi / 448 * (1 + 2 * U32)).clamp_min(2.0 ** -126)) & (s >= (lo / 448 * (1 - 2 * U32)).clamp_min(2.0 ** -126))).all()), what
    else:
        assert bool((448 * s >= lo).all()), what
        assert bool(((448 * s / 2 < hi) | (s == 2.0 ** -127)).all()), what
    sw = s.repeat_interleave(w // n, 1)
    got = codes.cpu().double() * sw
    # e4m3 below 2^-6 has steps of 2^-9; the largest code may stand for values that err lifts past it
    tol = HALF[torch.float8_e4m3fn] * (ref.abs() + err) + 2.0 ** -10 * sw + err * (1 + 2.0 ** -4)
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()))


def gated(gp, up):
    """silu(g) * u and its error bound from two (value, bound) pairs; |silu'| <= 1.1."""
    (g, eg), (u, eu) = gp, up
    silu = g / (1 + torch.exp(-g))
    y = silu * u
    return y, 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + 16 * U32 * y.abs()


def norm(x, residual, gamma, eps):
    """(stored stream, y, bound on y's fp32 error): the sum of squares is a
    chain of at most 64 fused multiply-adds a thread and 10 additions, halved
    by the square root; six roundings follow."""
    if residual is None:
        s = x
    else:
        s = (x.float() + residual.float()).to(residual.dtype)
    z = s.double()
    y = z / torch.sqrt((z * z).mean(1, keepdim=True) + float(np.float32(eps))) * gamma.double()
    return s, y, ((64 + 10) / 2 + 8) * U32 * y.abs()
