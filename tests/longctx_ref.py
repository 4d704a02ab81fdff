"""The long-context operators in 64 bits (torch on whatever device the inputs are), straight from
the definitions: codes are dequantised to keys and values and attended plainly; the error that
the kernels' 16-bit operands allow is computed from the same data."""
import math

import torch

D = 128
QJL = math.sqrt(math.pi / 2) / D


def bits(planes):
    """[..., 16] bytes -> [..., 128] bits, coordinate j at bit j % 8 of byte j // 8."""
    sh = torch.arange(8, device=planes.device, dtype=torch.uint8)
    return ((planes[..., None] >> sh) & 1).flatten(-2).long()


def tokens(cache, b, h, at):
    """Entries of a cache's arrays for tokens `at` of sequence b, head h: a function of
    (array, leading plane dims) -> rows."""
    pages = cache.pages
    if pages is None:
        return lambda t, planes: t[b, h][:, at] if planes else t[b, h][at]
    page = pages.block_table[b].long()[at // pages.page_tokens]
    slot = at % pages.page_tokens
    return lambda t, planes: t[page, h, :, slot].movedim(1, 0) if planes else t[page, h, slot]


def key_parts(k, kc, b, h, at):
    """(levels c, signs ±1, ‖x‖, ‖r‖) of tokens `at`, in 64 bits."""
    get = tokens(k, b, h, at)
    planes = get(k.idx, True)
    i = sum(bits(planes[p]) << p for p in range(planes.shape[0]))
    c = torch.tensor(kc.centroids, device=i.device)[i]
    return c, (2 * bits(get(k.sgn, False)) - 1).double(), get(k.xnorm, False).double(), \
        get(k.rnorm, False).double()


def value_parts(v, vc, b, h, at):
    get = tokens(v, b, h, at)
    if v.bits == 4:
        x = get(v.idx, False)
        j = torch.stack([x & 15, x >> 4], -1).flatten(-2).long()
    else:
        x = get(v.idx, True)
        j = sum(bits(x[p]) << p for p in range(v.bits))
    return torch.tensor(vc.centroids, device=j.device)[j], get(v.xnorm, False).double()


def attend(q, parts, kc, vc, scale=None, pairs=False):
    """Attention of query rows q [g, 128] over tokens given as (c, s, xn, rn, cv, vn); returns the
    rows and the standard deviation of the error (2-norm) that 16-bit operands allow.

    Roundings of the kernel, each uniform and off by at most u = eps(fp16) / 2 = 2^-11 relative, or
    with pairs of fp16 numbers (fp16 outputs) 2^-21 (standard deviation u / √3): y_j, z_j and a
    weight w_t, all independent; ρ_t, one for all of a token's signs; the levels, off by at most ε
    as scaled (the same for all tokens: taken at ε).  32-bit products and sums of a score: 2^-20 of
    its largest possible value.  A logit error δ_t moves the output by p_t·δ_t·(v_t − out): at
    most p_t·δ_t·(‖v_t‖ + ‖out‖).  Weights below 2^-14 of 2^8 (fp16 subnormals) add an absolute
    2^-25 each."""
    c, s, xn, rn, cv, vn = parts
    pi, sk = (torch.tensor(m, device=q.device) for m in (kc.pi, kc.s))
    vpi = torch.tensor(vc.pi, device=q.device)
    scale = scale or 1 / math.sqrt(D)
    q = q.double()
    if len(xn) == 0:
        return torch.zeros_like(q), torch.zeros(len(q), dtype=torch.float64, device=q.device)
    y, z = q @ pi.T, q @ sk.T
    main, sketch = xn * (y @ c.T), QJL * rn * (z @ s.T)
    p = torch.softmax(scale * (main + sketch), -1)
    v = vn[:, None] * (cv @ vpi)
    out = p @ v
    u = 2.0 ** (-21 if pairs else -11) / math.sqrt(3)
    ek, ev = level_error(kc), level_error(vc)
    var = scale ** 2 * ((u * xn) ** 2 * ((y ** 2) @ (c ** 2).T)
                        + (u * QJL * rn) ** 2 * (z ** 2).sum(-1, keepdim=True)
                        + (u * sketch) ** 2 + (ek * xn) ** 2 * ((y ** 2) @ (c ** 2).T)
                        + (2.0 ** -20 * (xn * y.norm(dim=-1, keepdim=True) * c.norm(dim=-1)
                                         + QJL * rn * z.norm(dim=-1, keepdim=True) * math.sqrt(D))) ** 2)
    size = vn + out.norm(dim=-1, keepdim=True)
    err = ((p * size) ** 2 * (var + u ** 2)).sum(-1).sqrt() + ev * out.norm(dim=-1)
    top = (p * vn).amax(-1)
    err = err + 2.0 ** -25 * top * math.sqrt(len(xn))
    # 32-bit sums: 2^-24 relative per addition of the accumulators' largest part
    err = err + 2.0 ** -22 * (p * vn).sum(-1)
    return out, err


def level_error(codec):
    """Largest relative error of the codec's levels held as fp16 after the best scale in [1, 2)."""
    c = torch.tensor(codec.centroids)
    c = c[c != 0]
    sg = 1 + torch.arange(1 << 16, dtype=torch.float64) / 65536
    x = sg[:, None] * c
    return float(((x.half().double() - x) / x).abs().amax(-1).min()) + 2.0 ** -24


def check_rows(got, ref, err, what):
    """Every row within eight standard deviations, and the output's own rounding."""
    step = torch.finfo(got.dtype).eps / 2
    off = (got.double() - ref).norm(dim=-1)
    most = 8 * err + step * ref.norm(dim=-1) + 1e-30
    if got.dtype == torch.float16:
        most = most + 2.0 ** -25 * math.sqrt(D)     # subnormal outputs
    bad = ~(off <= most)
    assert not bad.any(), (f"{what}: {int(bad.sum())} rows off, first {bad.nonzero()[0].tolist()}, "
                           f"error {float(off[bad][0]):.3g} over {float(most[bad][0]):.3g}")
    return float((off / most).max())


# ------------------------------------------------------------------ blocks

def outward(x, up):
    """The bf16 nearest to x that is not below (up) or not above it."""
    y = x.to(torch.bfloat16)
    wrong = (y.double() < x.double()) if up else (y.double() > x.double())
    inf = torch.tensor(math.inf if up else -math.inf, dtype=torch.bfloat16, device=x.device)
    return torch.where(wrong, torch.nextafter(y.cpu(), inf.cpu()).to(x.device), y)


def bounds(x, pos, count, old):
    """Bounds [B, H, nb, 2, 128] after keys x [B, H, T, 128] were folded into `old` (NaN left out)."""
    new = old.clone()
    for b in range(x.shape[0]):
        p, n = int(pos[b]), int(count[b])
        for blk in range(p // 64, (p + n - 1) // 64 + 1 if n else 0):
            a, e = max(blk * 64 - p, 0), min((blk + 1) * 64 - p, n)
            t = x[b, :, a:e].double()
            lo = torch.where(t.isnan(), math.inf, t).amin(1)
            hi = torch.where(t.isnan(), -math.inf, t).amax(1)
            lo, hi = outward(lo, False), outward(hi, True)
            if blk * 64 < p:
                lo, hi = torch.minimum(lo, old[b, :, blk, 0]), torch.maximum(hi, old[b, :, blk, 1])
            new[b, :, blk, 0], new[b, :, blk, 1] = lo, hi
    return new


def select(q, bnd, n, keep, first, last):
    """Kept blocks of one (sequence, KV head): q [g, 128], bounds [nb, 2, 128], n blocks."""
    if n <= keep:
        return list(range(n)) + [-1] * (keep - n)
    t = q.double()[:, None]
    lo, hi = bnd[:n, 0].double(), bnd[:n, 1].double()
    s = torch.where(t < 0, t * lo, t * hi).sum(-1)
    s = torch.where(s.isnan(), -math.inf, s).amax(0).tolist()
    forced = set(range(first)) | set(range(n - last, n))
    rest = sorted((i for i in range(n) if i not in forced), key=lambda i: (-s[i], i))
    return sorted(forced | set(rest[:keep - len(forced)]))
