"""Float64 reference of the low-rank adapter calls, request by request, with
the magnitudes that bound a correct result's distance from it."""
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# u = A x is held in fp32 and enters the second product as two storage-type
# halves: what they lose relative to the largest u they are scaled by.  bf16:
# the first half truncates (under 2^-7), the second rounds (2^-8 of that).
# f16: 2^-11 each, and 2^-25 of the scale where the second is subnormal.
SPLIT = {"f32": 0.0, "f16": 2.0 ** -21, "bf16": 2.0 ** -15}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}


def mm(a, b):
    return torch.mm(a.contiguous(), b.contiguous())


class Case:
    """Inputs of one call on `device`; lengths are the requests' tokens."""

    def __init__(self, dt, lengths, adapter, n, R, n_in, n_out, ranks=None, seed=0, device="cuda",
                 lead=0, tail=0, scaled=True, pad=0):
        g = torch.Generator().manual_seed(seed)

        def normal(shape, std):
            return (torch.randn(shape, generator=g) * std).to(DT[dt]).to(device)

        def matrix(rows, cols, std):
            # rows apart by more than their length, starting off the allocation's start
            return normal((rows, cols + 2 * pad), std)[:, pad:pad + cols]

        self.dt, self.n, self.R, self.n_in, self.n_out = dt, n, R, n_in, n_out
        self.T = lead + sum(lengths) + tail
        off = [lead]
        for length in lengths:
            off.append(off[-1] + length)
        self.off, self.ad = off, list(adapter)
        self.offsets = torch.tensor(off, dtype=torch.int32, device=device)
        self.adapter = torch.tensor(self.ad, dtype=torch.int32, device=device)
        self.rk = [R] * n if ranks is None else list(ranks)
        self.ranks = None if ranks is None else torch.tensor(self.rk, dtype=torch.int32,
                                                             device=device)
        self.scale = (torch.rand(n, generator=g) * 1.5 + 0.5).to(device) if scaled else None
        self.A = normal((n, R, n_in), n_in ** -0.5)
        self.B = normal((n, n_out, R), R ** -0.5)
        self.xt = matrix(n_in, self.T, 1.0)
        self.yt = matrix(n_out, self.T, 1.0)
        self.dyt = matrix(n_out, self.T, 1.0)
        self.W = matrix(n_out, n_in, n_in ** -0.5)

    def args(self):
        return (self.xt, self.A, self.B, self.offsets, self.adapter, self.scale, self.ranks)

    def runs(self):
        """(token slice, adapter, rank, scale) of each request that has an adapter."""
        for i, a in enumerate(self.ad):
            if 0 <= a < self.n and self.off[i] < self.off[i + 1]:
                k = min(max(self.rk[a], 0), self.R)
                if k:
                    s = 1.0 if self.scale is None else float(self.scale[a])
                    yield slice(self.off[i], self.off[i + 1]), a, k, s


def sum_error(*terms):
    """fp32 sums in any order: at most one 2^-24 of the terms' magnitude a step."""
    return (sum(terms) + 8) * 2.0 ** -24


def forward(c, base, base_mag, base_terms=0):
    """(y, bound) for y = base + adapters; base in float64."""
    y, mag = base.clone(), base_mag.clone()
    for t, a, k, s in c.runs():
        x, A, B = c.xt[:, t].double(), c.A[a, :k].double(), c.B[a, :, :k].double()
        y[:, t] += s * mm(B, mm(A, x))
        big = mm(A.abs(), x.abs()).amax(0, keepdim=True)  # over ranks: f16's scale
        mag[:, t] += s * B.abs().sum(1, keepdim=True) * big
    eps = torch.finfo(DT[c.dt]).eps / 2
    rel = sum_error(c.n_in, c.R, base_terms) + SPLIT[c.dt]
    return y, eps * y.abs() * (1 + 2 * rel) + rel * mag * (1 + eps) + TINY[c.dt]


def add(c):
    base = c.yt.double()
    return forward(c, base, base.abs())


def project(c):
    W, x = c.W.double(), c.xt.double()
    return forward(c, mm(W, x), mm(W.abs(), x.abs()), c.n_in)


def backward(c):
    """[(dx, bound), (dA, bound), (dB, bound)]"""
    dx = torch.zeros(c.n_in, c.T, dtype=torch.float64, device=c.xt.device)
    dA, dB = torch.zeros_like(c.A, dtype=torch.float64), torch.zeros_like(c.B, dtype=torch.float64)
    mx, mA, mB = torch.zeros_like(dx), torch.zeros_like(dA), torch.zeros_like(dB)
    # f16's scale of a rank's du (u) is its largest over up to 32 tokens of the
    # adapter: bounded by the largest over all of them
    big_u, big_du = {}, {}
    for t, a, k, s in c.runs():
        x, dy = c.xt[:, t].double(), c.dyt[:, t].double()
        A, B = c.A[a, :k].double(), c.B[a, :, :k].double()
        u = s * mm(A.abs(), x.abs()).amax(1)
        du = s * mm(B.abs().t(), dy.abs()).amax(1)
        big_u[a] = torch.maximum(big_u[a], u) if a in big_u else u
        big_du[a] = torch.maximum(big_du[a], du) if a in big_du else du
    for t, a, k, s in c.runs():
        x, dy = c.xt[:, t].double(), c.dyt[:, t].double()
        A, B = c.A[a, :k].double(), c.B[a, :, :k].double()
        u, du = s * mm(A, x), s * mm(B.t(), dy)
        dx[:, t] = mm(A.t(), du)
        dA[a, :k] += mm(du, x.t())
        dB[a, :, :k] += mm(dy, u.t())
        mdu = s * mm(B.abs().t(), dy.abs())
        mx[:, t] = A.abs().sum(0)[:, None] * mdu.amax(0, keepdim=True)
        mA[a, :k] += big_du[a][:, None] * x.abs().sum(1)[None, :]
        mB[a, :, :k] += dy.abs().sum(1)[:, None] * big_u[a][None, :]
    eps = torch.finfo(DT[c.dt]).eps / 2
    out = []
    for v, m, terms in ((dx, mx, (c.n_out, c.R)), (dA, mA, (c.n_out, c.T)),
                        (dB, mB, (c.n_in, c.T))):
        rel = sum_error(*terms) + SPLIT[c.dt]
        out.append((v, eps * v.abs() * (1 + 2 * rel) + rel * m * (1 + eps) + TINY[c.dt]))
    return out


def check(got, want, what=""):
    ref, bound = want
    assert got.shape == ref.shape, what
    off = (got.double() - ref).abs() - bound
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0.0, f"{what}: {int((off > 0).sum())} values outside their bound, by {worst:.3g}"
    assert torch.isfinite(got).all(), what
