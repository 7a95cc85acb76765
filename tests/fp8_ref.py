"""Plain fp64 forms (torch) of the operators on rows in 8 bits, written from
their formulas, for the tests of the GPU kernels."""
import math

import torch

F64 = torch.float64
U24 = 2.0 ** -24   # half a step of fp32
U8 = 2.0 ** -8     # half a step of bf16
U4 = 2.0 ** -4     # half a step of E4M3
NAN_CODE = 0x7F


def e4m3_table():
    """The values of the 256 codes, by the format's definition (code 0x7f and 0xff: NaN)."""
    out = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.nan if (c & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out.append(-v if c & 128 else v)
    return torch.tensor(out, dtype=F64)


TABLE = e4m3_table()


def encode(v):
    """E4M3 codes of fp64 values, to nearest, ties to the even code; NaN of what is not finite.  Values are within
    448 + half a step."""
    mags = TABLE[:127].to(v.device)
    a = v.abs().contiguous()
    hi = torch.searchsorted(mags, a).clamp(1, 126)
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = torch.where(torch.isfinite(v), code, NAN_CODE)
    return (code + 128 * torch.signbit(v).to(code.dtype)).to(torch.uint8)


def same_codes(a, b):
    """Equal codes, any NaN for any NaN (its sign says nothing)."""
    return torch.equal(torch.where((a & 127) == 127, 127, a), torch.where((b & 127) == 127, 127, b))


def blocks(v):
    pad = -v.shape[-1] % 128
    return torch.cat((v, v.new_zeros(*v.shape[:-1], pad)), -1).unflatten(-1, (-1, 128))


def spread(s, n):
    return s.repeat_interleave(128, -1)[..., :n]


def quantize(x):
    """(codes, E8M0 codes) of bf16 rows: the least power of two that brings the largest finite value to 448."""
    d = x.double()
    amax = blocks(torch.where(torch.isfinite(d), d, 0.0)).abs().amax(-1)
    e = torch.full_like(amax, -126)
    for _ in range(260):
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    return encode(d * torch.exp2(-spread(e, x.shape[-1]))), (e + 127).to(torch.uint8)


def rows(q, sf):
    """fp64 values of quantised rows."""
    return TABLE.to(q.device)[q.long()] * spread(torch.exp2(sf.double() - 127), q.shape[-1])


def halves(x):
    """The quantisation of each half of the rows, side by side."""
    I = x.shape[-1] // 2
    a, b = quantize(x[:, :I]), quantize(x[:, I:])
    return torch.cat((a[0], b[0]), 1), torch.cat((a[1], b[1]), 1)


def halves_rows(q, sf):
    I, nb = q.shape[-1] // 2, sf.shape[-1] // 2
    return torch.cat((rows(q[:, :I], sf[:, :nb]), rows(q[:, I:], sf[:, nb:])), 1)


def quantize_weight(w):
    """(codes, fp32 scales) of bf16 [N, K]: fp32 quotients, as the header defines them."""
    N, K = w.shape
    f = w.float()
    fin = torch.where(torch.isfinite(f), f, 0.0).abs()
    pad = torch.nn.functional.pad(fin, (0, -K % 128, 0, -N % 128))
    amax = pad.unflatten(1, (-1, 128)).amax(2).unflatten(0, (-1, 128)).amax(1)
    sf = (amax / 448).clamp(min=2.0 ** -126)
    return encode((f / spread_weight(sf, N, K)).double().clamp(-448, 448) if bool(torch.isfinite(f).all()) else
                  torch.where(torch.isfinite(f), (f / spread_weight(sf, N, K)).double().clamp(-448, 448),
                              f.double())), sf


def spread_weight(sf, N, K):
    return sf.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def weights(q, sf):
    return TABLE.to(q.device)[q.long()] * spread_weight(sf.double(), *q.shape)


def product_bound(x, w):
    """What the matrix instruction may lose of each output of x w^T (fp64 values): 2^-13 of the power of two of the
    largest of 8 consecutive products, eight times; x is a few rows."""
    out = []
    for r in x:
        p = (r * w).abs()
        out.append(torch.nn.functional.pad(p, (0, -p.shape[1] % 8)).unflatten(1, (-1, 8)).amax(2).sum(1))
    return 8 * 2.0 ** -13 * torch.stack(out)


def act(kind, g, u, alpha=1.0, beta=0.0, limit=math.inf):
    """(f, f', up, up') of the gated activations, fp64."""
    if kind == "geglu":
        c = math.sqrt(2 / math.pi)
        z = c * (g + 0.044715 * g ** 3)
        t = torch.tanh(z)
        sech2 = 1 / torch.cosh(z.clamp(-300, 300)) ** 2
        return (0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * sech2 * c * (1 + 3 * 0.044715 * g * g), u,
                torch.ones_like(u))
    gc, uc = g.clamp(max=limit), u.clamp(-limit, limit)
    s = torch.sigmoid(alpha * gc)
    return (gc * s, s * (1 + alpha * gc * torch.sigmoid(-alpha * gc)) * (g <= limit), uc + beta,
            (u.abs() <= limit).double())
