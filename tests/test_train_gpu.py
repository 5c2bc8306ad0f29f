"""The training-side operators against their formulas in 64 bits.

Tolerances count roundings: u = 2^-24 for a 32-bit operation, h = 2^-8 for a
bf16 store (half a step). Sums of n terms are held to DEPTH * u times the sum
of the terms' absolute values, DEPTH = 256 being more than the longest chain of
additions a result goes through at these sizes (a lane's own terms, the lanes
of a workgroup, the chunks and images).
"""
import pytest
import torch

import convolution_conv2d_nhwc_amd as conv
from convolution_conv2d_nhwc_amd import train

pytestmark = pytest.mark.gpu

U, HALF, DEPTH = 2.0 ** -24, 2.0 ** -8, 256
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check(got, ref, tol, what):
    got = got.double().cpu()
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %g against %g" % (
        what, int(bad.sum()), bad.numel(), float((got - ref).abs()[bad].max()), float((tol + 0 * ref)[bad].max()))


# ------------------------------------------------------------------ group norm --

def act_of(z, act):
    """act(z) and its slope."""
    q = torch.sigmoid(z)
    if act == "silu":
        return z * q, q + z * q * (1 - q)
    if act == "mish":
        t = torch.tanh(torch.nn.functional.softplus(z))
        return z * t, t + z * q * (1 - t * t)
    if act == "relu":
        return z.clamp_min(0), (z > 0).double()
    if act == "relu6":
        return z.clamp(0, 6), ((z > 0) & (z < 6)).double()
    return z, torch.ones_like(z)


def norm_ref(x, groups, gamma, beta, act, eps, dy=None):
    """Outputs of the formula in 64 bits, each with its tolerance."""
    n, h, w, c = x.shape
    cg = c // groups
    x = x.double().reshape(n, h * w, groups, cg)
    g = (gamma.double() if gamma is not None else torch.ones(c, dtype=torch.float64)).view(1, 1, groups, cg)
    b = (beta.double() if beta is not None else torch.zeros(c, dtype=torch.float64)).view(1, 1, groups, cg)
    mean = x.mean((1, 3), keepdim=True)
    var = ((x - mean) ** 2).mean((1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xh = (x - mean) * rstd
    z = g * xh + b
    y, slope = act_of(z, act)
    # xhat: the mean is off by up to a few u of the largest value, rstd by a few u
    top = x.abs().amax((1, 3), keepdim=True) * rstd
    exh = 16 * U * (xh.abs() + top)
    ez = g.abs() * exh + 4 * U * (z.abs() + b.abs())
    # every activation's slope and the slope's slope are below 1.1; their evaluation costs 16 u
    ey = 1.1 * ez + 16 * U * (y.abs() + z.abs())
    out = {"y": (y.reshape(n, h, w, c), ey.reshape(n, h, w, c)),
           "stats": (torch.stack([mean.flatten(), rstd.flatten()], 1).view(n, groups, 2),
                     torch.stack([(16 * U * x.abs().amax((1, 3), keepdim=True)).flatten(),
                                  (rstd * 16 * U * (1 + top)).flatten()], 1).view(n, groups, 2))}
    if dy is None:
        return out
    dy = dy.double().reshape(n, h * w, groups, cg)
    dz = dy * slope
    # where z is next to a kink the slope may fall on either side
    kink = torch.zeros_like(z)
    if act in ("relu", "relu6"):
        kink = (z.abs() <= ez).double()
    if act == "relu6":
        kink = kink + ((z - 6).abs() <= ez).double()
    edz = dy.abs() * (1.1 * ez + 16 * U + kink)
    dbeta, sdb = dz.sum((0, 1)), dz.abs().sum((0, 1))
    dgamma, sdg = (dz * xh).sum((0, 1)), (dz * xh).abs().sum((0, 1))
    edb = DEPTH * U * sdb + edz.sum((0, 1))
    edg = DEPTH * U * sdg + (edz * xh.abs() + dz.abs() * exh).sum((0, 1))
    t = g * dz
    et = g.abs() * edz
    m1, m2 = t.mean((1, 3), keepdim=True), (t * xh).mean((1, 3), keepdim=True)
    em1 = DEPTH * U * t.abs().mean((1, 3), keepdim=True) + et.mean((1, 3), keepdim=True)
    em2 = DEPTH * U * (t * xh).abs().mean((1, 3), keepdim=True) + (et * xh.abs() + t.abs() * exh).mean((1, 3), keepdim=True)
    dx = rstd * (t - m1 - xh * m2)
    edx = rstd * (et + em1 + xh.abs() * em2 + exh * m2.abs()) + 16 * U * rstd * (t.abs() + m1.abs() + (xh * m2).abs()) \
        + 4 * U * top * dx.abs()
    out.update(dx=(dx.reshape(n, h, w, c), edx.reshape(n, h, w, c)), dgamma=(dgamma.reshape(c), edg.reshape(c)),
               dbeta=(dbeta.reshape(c), edb.reshape(c)))
    return out


def store_tol(ref, tol, dtype):
    return tol + (HALF * (ref.abs() + tol) if dtype == "bf16" else 0)


def run_norm(x, groups, gamma, beta, act, eps=1e-5, dy=None):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    n = x.shape[0]
    xd = x if x.is_cuda else x.cuda()
    stats = torch.full((n, groups, 2), float("nan"), device="cuda")
    y = torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda")
    conv.group_norm(xd, groups, dev(gamma), dev(beta), eps=eps, act=act, y=y, stats=stats)
    out = {"y": y, "stats": stats}
    if dy is not None:
        c = x.shape[3]
        dx = torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda")
        dg, db = (torch.full((c,), float("nan"), device="cuda") for _ in range(2))
        conv.group_norm_grad(dev(dy), xd, stats, dev(gamma), dev(beta), act=act, dx=dx, dgamma=dg, dbeta=db)
        out.update(dx=dx, dgamma=dg, dbeta=db)
    return out


def check_norm(x, groups, gamma, beta, act, dtype, eps=1e-5, dy=None):
    ref = norm_ref(x.cpu(), groups, gamma, beta, act, eps, dy)
    got = run_norm(x, groups, gamma, beta, act, eps, dy)
    for k, (r, t) in ref.items():
        check(got[k], r, store_tol(r, t, dtype) if k in ("y", "dx") else t, k)


# n, h, w, c, groups
NORM_SHAPES = [
    (1, 1, 1, 1, 1), (1, 1, 1, 32, 4), (2, 1, 3, 7, 7), (1, 5, 5, 6, 1), (3, 2, 2, 5, 1),
    (1, 20, 20, 512, 32),     # narrow tiles, one launch
    (2, 9, 7, 40, 8),         # groups of 5: vectors that straddle groups
    (1, 13, 11, 36, 12),      # groups of 3
    (4, 3, 5, 1100, 1),       # a group of several tiles
    (1, 40, 33, 1040, 2),     # the same with chunks
    (2, 45, 39, 64, 4),       # one launch of 1024 lanes
    (1, 150, 149, 24, 3),     # streamed, ragged chunks
    (2, 70, 71, 10, 2),       # streamed, groups of 5
    (17, 4, 4, 16, 16),       # a channel a group
    (1, 300, 7, 3, 3), (1, 2, 2, 512, 1),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_group_norm(shape, dtype):
    n, h, w, c, groups = shape
    g = gen(h * w + c)
    act = ["none", "relu", "relu6", "mish", "silu"][(h + c) % 5]
    x = (torch.randn((n, h, w, c), generator=g) * (0.5 + torch.rand(c, generator=g)) + torch.randn(c, generator=g)).to(DT[dtype])
    dy = torch.randn((n, h, w, c), generator=g).to(DT[dtype])
    gamma, beta = 1 + 0.3 * torch.randn(c, generator=g), 0.3 * torch.randn(c, generator=g)
    # a single value's group has no spread: eps keeps the formula's slope tame
    check_norm(x, groups, gamma, beta, act, dtype, eps=1e-5 if h * w * c // groups > 1 else 1.0, dy=dy)


@pytest.mark.parametrize("act", ["none", "relu", "relu6", "mish", "silu"])
@pytest.mark.parametrize("affine", ["both", "gamma", "beta", "none"])
def test_group_norm_activations_without_affine(act, affine):
    g = gen(3)
    x = 3 * torch.randn((2, 8, 9, 24), generator=g)
    dy = torch.randn(x.shape, generator=g)
    gamma = 4 * torch.randn(24, generator=g) if affine in ("both", "gamma") else None  # z of a wide range
    beta = 4 * torch.randn(24, generator=g) if affine in ("both", "beta") else None
    check_norm(x, 6, gamma, beta, act, "f32", dy=dy)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("c,pitch,off", [(60, 100, 20), (16, 40, 8), (24, 25, 1), (8, 64, 3), (12, 12, 0)])
def test_group_norm_reads_a_channel_slice(dtype, c, pitch, off):
    g = gen(c + pitch)
    wide = torch.randn((2, 6, 7, pitch), generator=g).to(DT[dtype]).cuda()
    x = wide[..., off:off + c]
    dy = torch.randn((2, 6, 7, c), generator=g).to(DT[dtype])
    gamma = torch.randn(c, generator=g)
    check_norm(x, 4, gamma, None, "silu", dtype, dy=dy)


@pytest.mark.parametrize("shape", [(1, 12, 12, 16, 2), (1, 200, 180, 8, 2)])
def test_group_norm_large_offset_costs_no_digits(shape):
    n, h, w, c, groups = shape
    x = torch.randn((n, h, w, c), generator=gen(1)) + 4096.0
    check_norm(x, groups, None, None, "none", "f32")


def test_group_norm_constant_map_and_zero_upstream():
    x = torch.full((2, 5, 5, 8), 3.0)
    out = run_norm(x, 2, None, None, "silu", dy=torch.zeros_like(x))
    assert torch.equal(out["y"].cpu(), torch.zeros_like(x))
    for k in ("dx", "dgamma", "dbeta"):
        assert not out[k].any()


@pytest.mark.parametrize("shape", [(2, 6, 6, 32, 4), (2, 150, 150, 16, 4)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_group_norm_keeps_nan_in_its_group(shape, value):
    n, h, w, c, groups = shape
    g = gen(5)
    x = torch.randn((n, h, w, c), generator=g)
    dy = torch.randn(x.shape, generator=g)
    for act in ("relu", "relu6", "mish", "silu"):
        clean = run_norm(x, groups, None, None, act, dy=dy)
        bad = x.clone()
        bad[1, 2, 3, 0] = value
        out = run_norm(bad, groups, None, None, act, dy=dy)
        cg = c // groups
        for k in ("y", "dx"):
            assert torch.isnan(out[k][1, ..., :cg]).all() or value != value and torch.isnan(out[k][1, ..., :cg]).all()
            assert torch.equal(out[k][0], clean[k][0]) and torch.equal(out[k][1, ..., cg:], clean[k][1, ..., cg:])
        assert torch.isnan(out["dgamma"][:cg]).all()
        assert torch.equal(out["dgamma"][cg:], clean["dgamma"][cg:]) and torch.equal(out["dbeta"][cg:], clean["dbeta"][cg:])


@pytest.mark.parametrize("act", ["mish", "silu", "none"])
def test_group_norm_gradient_against_differences(act):
    """(total(p + s d) - total(p - s d)) / 2 s of the 64-bit formula is the
    gradient along d to s^2 (third derivatives of order one)."""
    g = gen(11)
    x, dy = torch.randn((2, 4, 5, 12), generator=g), torch.randn((2, 4, 5, 12), generator=g)
    gamma, beta = torch.randn(12, generator=g), torch.randn(12, generator=g)
    out = run_norm(x, 3, gamma, beta, act, dy=dy)
    s = 1e-4
    for i, name in enumerate(("dx", "dgamma", "dbeta")):
        d = torch.randn((x, gamma, beta)[i].shape, generator=g).double()
        total = []
        for sign in (1, -1):
            p = [x.double(), gamma.double(), beta.double()]
            p[i] = p[i] + sign * s * d
            total.append(float((norm_ref(p[0], 3, p[1], p[2], act, 1e-5)["y"][0] * dy.double()).sum()))
        want = (total[0] - total[1]) / (2 * s)
        got = float((out[name].cpu().double() * d).sum())
        assert abs(got - want) <= 1e-4 * float((out[name].cpu().double() * d).abs().sum() + 1), (name, got, want)


# ------------------------------------------------------------------- head loss --

def loss_ref(x, w, labels, weights):
    """Formula in 64 bits and tolerances. x, w bf16 on any device."""
    rows, (v, c) = x.shape[0], w.shape
    kept = (labels >= 0) & (labels < v)
    at = torch.where(kept, labels, 0).long()
    xd, wd = torch.where(kept[:, None], x.double(), 0.0), w.double()
    k = weights.double() if weights is not None else torch.full((rows,), 1.0 / max(1, int(kept.sum())), dtype=torch.float64, device=x.device)
    k = torch.where(kept, k, 0.0)
    s = xd @ wd.t()
    lse = torch.logsumexp(s, 1)
    sl = s.gather(1, at[:, None])[:, 0]
    loss = torch.where(kept, lse - sl, 0.0)
    # a logit: chains of c / 32 products of 32, four of them added
    es = (c / 32 + 36) * U * (xd.abs() @ wd.abs().t()).amax(1)
    el = torch.where(kept, 2 * es + 16 * U * (lse.abs() + sl.abs() + 1), 0.0)
    p = torch.exp(s - lse[:, None])
    hot = torch.zeros_like(p).scatter_(1, at[:, None], 1.0)
    g = (p - hot) * k[:, None]
    # off by the logits' error; rounded to bf16 but for the label's entry, whose rest keeps 8 bits more
    eg = k.abs()[:, None] * p * (4 * es + 32 * U)[:, None] + 4 * U * g.abs()
    er = HALF * (g.abs() + eg) * (1 - hot) + HALF * HALF * (g.abs() + eg) * hot
    dx, dw = g @ wd, g.t() @ xd
    depth = DEPTH * U
    edx = (er + eg + depth * g.abs()) @ wd.abs()
    edw = (er + eg + depth * g.abs()).t() @ xd.abs()
    total, et = (loss * k).sum(), (el * k.abs()).sum() + 4 * U * (loss * k).abs().sum()
    return {"total": (total, et), "loss": (loss, el), "dx": (dx, edx + HALF * (dx.abs() + edx)),
            "dw": (dw, edw + HALF * (dw.abs() + edw))}


def run_loss(x, w, labels, weights):
    nan = lambda *s, **k: torch.full(s, float("nan"), device="cuda", **k)  # noqa: E731
    total, loss = nan(), nan(*labels.shape)
    dx, dw = nan(*x.shape, dtype=torch.bfloat16), nan(*w.shape, dtype=torch.bfloat16)
    conv.head_loss_grad(x, w, labels, weights, loss=loss, total=total, dx=dx, dw=dw)
    t2, l2 = conv.head_loss(x, w, labels, weights)
    bits = lambda t: t.view(torch.int32)  # noqa: E731  (NaN equal to itself)
    assert torch.equal(bits(l2), bits(loss)) and torch.equal(bits(t2), bits(total))
    return {"total": total, "loss": loss, "dx": dx, "dw": dw}


def loss_case(rows, c, v, seed=0, scale=2.0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed + rows * 7 + c)
    w = torch.randn((v, c), generator=g, device=device) * (scale / c ** 0.5)
    labels = torch.randint(0, v, (rows,), generator=g, device=device)
    x = torch.randn((rows, c), generator=g, device=device) + w[labels]
    return x.bfloat16(), w.bfloat16(), labels, g


def check_loss(x, w, labels, weights):
    got = run_loss(x, w, labels, weights)
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    for k, (r, t) in loss_ref(cpu(x), cpu(w), cpu(labels), cpu(weights)).items():
        check(got[k], r, t, k)


LOSS_SHAPES = [
    (1, 8, 1), (1, 1, 2), (3, 5, 7), (1, 64, 100), (5, 107, 316), (125, 64, 1000), (64, 56, 64), (65, 72, 129),
    (513, 40, 70),       # rows past the one-workgroup reduction
    (40, 33, 6001),      # classes past it
    (300, 200, 2500), (129, 1000, 257),
    (2000, 24, 1030),    # long reductions over rows
    (700, 130, 12000),   # long reductions over classes: split
]


@pytest.mark.parametrize("shape", LOSS_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_head_loss(shape):
    x, w, labels, _ = loss_case(*shape)
    check_loss(x, w, labels, None)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("shape", [(50, 32, 90), (700, 100, 1100)])
def test_head_loss_left_out_rows_and_weights(shape, dtype):
    x, w, labels, g = loss_case(*shape)
    labels[::3] = -100
    labels[1] = shape[2]        # one past the last
    labels[4] = -1
    x[::3] = float("nan")       # never used
    x[1] = float("inf")
    weights = torch.randn(shape[0], generator=g, device="cuda")  # of either sign
    weights[5] = 0.0
    check_loss(x, w, labels.to(dtype), weights)
    check_loss(x, w, labels.to(dtype), None)


@pytest.mark.parametrize("shape", [(7, 16, 33), (600, 64, 400)])
def test_head_loss_all_rows_left_out(shape):
    x, w, labels, _ = loss_case(*shape)
    out = run_loss(x, w, torch.full_like(labels, -100), None)
    for k in out:
        assert not out[k].any(), k


def test_head_loss_far_labels_do_not_wrap():
    x, w, labels, _ = loss_case(6, 16, 20)
    far = labels.clone()
    far[0], far[1], far[2] = 2 ** 32 + 3, -2 ** 32 + 3, 2 ** 63 - 1  # the low words are classes
    out = run_loss(x, w, far, None)
    assert not out["loss"][:3].any() and not out["dx"][:3].any()
    check_loss(x, w, far, None)


@pytest.mark.parametrize("rows,classes", [(3000, 64), (2500, 300), (100, 1000)])
def test_head_loss_one_label_for_all(rows, classes):
    """Every row's label in one tile: the label terms come in several lists."""
    x, w, labels, _ = loss_case(rows, 32, classes)
    check_loss(x, w, torch.full_like(labels, 5), None)


@pytest.mark.parametrize("off", [1, 2, 4])
def test_head_loss_unaligned_operands(off):
    rows, c, v = 70, 32, 200
    x, w, labels, _ = loss_case(rows, c, v)
    xb = torch.zeros(rows * c + 8, dtype=torch.bfloat16, device="cuda")
    wb = torch.zeros(v * c + 8, dtype=torch.bfloat16, device="cuda")
    xb[off:off + rows * c], wb[off:off + v * c] = x.flatten(), w.flatten()
    check_loss(xb[off:off + rows * c].view(rows, c), wb[off:off + v * c].view(v, c), labels, None)


def test_head_loss_large_logits():
    """Logits of thousands: no overflow, certain rows lose nothing."""
    x, w, labels, _ = loss_case(40, 64, 500, scale=200.0)
    check_loss((x * 16).bfloat16(), w, labels, None)


def test_head_loss_nan_row_stays_in_its_row():
    x, w, labels, _ = loss_case(90, 48, 300)
    clean = run_loss(x, w, labels, None)
    x[7, 3] = float("nan")
    out = run_loss(x, w, labels, None)
    assert torch.isnan(out["loss"][7]) and torch.isnan(out["total"]) and torch.isnan(out["dx"][7]).all()
    keep = torch.arange(90) != 7
    assert torch.equal(out["loss"][keep], clean["loss"][keep]) and torch.equal(out["dx"][keep], clean["dx"][keep])


def test_head_loss_on_a_map_and_ohwi_weights():
    x, w, labels, _ = loss_case(2 * 5 * 7, 24, 60)
    total, loss, dx, dw = conv.head_loss_grad(x.view(2, 5, 7, 24), w.view(60, 1, 1, 24), labels.view(2, 5, 7))
    flat = run_loss(x, w, labels, None)
    assert loss.shape == (2, 5, 7) and dx.shape == (2, 5, 7, 24) and dw.shape == (60, 1, 1, 24)
    assert torch.equal(total, flat["total"]) and torch.equal(dx.view(-1, 24), flat["dx"])
    assert torch.equal(dw.view(60, 24), flat["dw"]) and torch.equal(loss.flatten(), flat["loss"])


@pytest.mark.parametrize("rows,c,v", [(70000, 16, 4500), (4100, 40, 70001)])
def test_head_loss_in_pieces_of_the_classes(rows, c, v):
    """More than 2^28 entries of g: the gradient runs in pieces. The reference,
    in 64 bits on the device, a block of rows at a time."""
    x, w, labels, g = loss_case(rows, c, v)
    labels[::5] = -100
    got = run_loss(x, w, labels, None)
    weights = torch.full((rows,), 1.0 / int((labels >= 0).sum()), device="cuda")
    dw = torch.zeros((v, c), dtype=torch.float64, device="cuda")
    edw = torch.zeros_like(dw)
    step = (1 << 26) // v
    for i in range(0, rows, step):
        sl = slice(i, i + step)
        r = loss_ref(x[sl], w, labels[sl], weights[sl])
        for k in ("loss", "dx"):
            assert ((got[k][sl].double() - r[k][0]).abs() <= r[k][1]).all(), (k, i)
        dw += r["dw"][0]
        edw += r["dw"][1]
    assert ((got["dw"].double() - dw).abs() <= edw + HALF * dw.abs()).all()


def test_head_loss_gradient_against_differences():
    x, w, labels, g = loss_case(30, 16, 50)
    weights = torch.rand(30, generator=g, device="cuda")
    out = run_loss(x, w, labels, weights)
    args = [x.cpu().double(), w.cpu().double()]
    s = 1e-4
    for i, name in enumerate(("dx", "dw")):
        d = torch.randn(args[i].shape, generator=gen(2)).double()
        total = []
        for sign in (1, -1):
            p = list(args)
            p[i] = p[i] + sign * s * d
            total.append(float(loss_ref(p[0], p[1], labels.cpu(), weights.cpu())["total"][0]))
        want = (total[0] - total[1]) / (2 * s)
        got = float((out[name].cpu().double() * d).sum())
        # each entry is a bf16 number of two roundings' error at most
        assert abs(got - want) <= 2 * HALF * float((out[name].cpu().double() * d).abs().sum())


# ------------------------------------------------------------ orthogonalisation --

def ortho_ref(g, steps=5, coeffs=train.MUON_COEFFS, eps=1e-7):
    a, b, c = coeffs
    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-1, -2)
    x = x / (x.pow(2).sum((-1, -2), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        p = x @ x.transpose(-1, -2)
        x = a * x + (b * p + c * (p @ p)) @ x
    return (x.transpose(-1, -2) if tall else x).contiguous()


def check_ortho(got, ref, steps=5):
    """In the 2-norm: the bf16 store is off by half a step, each of a step's
    three products by the half step of its fp16 operands (2^-11)."""
    got = got.double().cpu()
    assert got.shape == ref.shape
    err = (got - ref).flatten(-2).norm(dim=-1)
    assert (err <= (HALF + 3 * steps * 2.0 ** -11) * ref.flatten(-2).norm(dim=-1)).all(), err


ORTHO_SHAPES = [(1, 1, 1), (2, 1, 5), (3, 8, 8), (1, 7, 1), (2, 33, 100), (1, 64, 576), (1, 64, 1024), (2, 500, 17),
                (1, 1024, 64), (1, 63, 1023), (2, 64, 1025), (2, 65, 70), (6, 200, 50), (1, 129, 513), (3, 300, 100),
                (1, 250, 1000), (1, 700, 900), (1, 1000, 1900)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", ORTHO_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_orthogonalize(shape, dtype):
    b, m, n = shape
    g = gen(m + n)
    r = max(1, min(m, n) // 8)
    x = (1e-3 * (torch.randn(shape, generator=g) + torch.randn((b, m, r), generator=g) @ torch.randn((b, r, n), generator=g))).to(DT[dtype])
    out = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    conv.orthogonalize(x.cuda(), out=out)
    check_ortho(out, ortho_ref(x))


@pytest.mark.parametrize("shape", [(40, 90), (130, 200)])
@pytest.mark.parametrize("steps", [1, 2, 8])
def test_orthogonalize_steps_and_coefficients(shape, steps):
    x = torch.randn(shape, generator=gen(steps))
    coeffs = (2.0, -1.5, 0.5)
    check_ortho(conv.orthogonalize(x.cuda(), steps=steps, coeffs=coeffs), ortho_ref(x, steps, coeffs), steps)


@pytest.mark.parametrize("shape", [(48, 80), (150, 90)])
@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_orthogonalize_any_scale(shape, scale):
    """The update does not depend on the gradient's scale, whose squares leave
    the 32-bit range here."""
    x = torch.randn(shape, generator=gen(4))
    check_ortho(conv.orthogonalize((x * scale).cuda(), eps=0.0), ortho_ref(x * scale, eps=0.0))


@pytest.mark.parametrize("shape", [(3, 30, 40), (3, 90, 130)])
def test_orthogonalize_zero_and_nan_matrices_in_a_batch(shape):
    x = torch.randn(shape, generator=gen(9))
    clean = conv.orthogonalize(x.cuda())
    x[0] = 0.0
    x[2, 3, 4] = float("nan")
    out = conv.orthogonalize(x.cuda())
    assert not out[0].any() and torch.equal(out[1], clean[1]) and torch.isnan(out[2].float()).all()


@pytest.mark.parametrize("shape", [(40, 91), (90, 131), (200, 70)])
@pytest.mark.parametrize("off", [1, 2])
def test_orthogonalize_unaligned(shape, off):
    m, n = shape
    x = torch.randn(shape, generator=gen(m))
    buf = torch.zeros(m * n + 4, device="cuda")
    buf[off:off + m * n] = x.flatten().cuda()
    out = torch.zeros(m * n + 8, dtype=torch.bfloat16, device="cuda")[off:off + m * n].view(m, n)
    conv.orthogonalize(buf[off:off + m * n].view(m, n), out=out)
    check_ortho(out, ortho_ref(x))
    assert torch.equal(out, conv.orthogonalize(x.cuda()))


def test_orthogonalize_ohwi_layer():
    g = torch.randn((96, 3, 3, 32), generator=gen(1))
    out = conv.orthogonalize(g.cuda())
    assert out.shape == g.shape
    check_ortho(out.view(96, -1), ortho_ref(g.view(96, -1)))


# --------------------------------------------------------- streams, graphs, scratch --

def all_calls(seed):
    """Calls of every operator on inputs of the seed, by name."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    d = {"x1": r(2, 10, 12, 64), "x2": r(1, 150, 150, 16).bfloat16(), "dy1": r(2, 10, 12, 64), "dy2": r(1, 150, 150, 16).bfloat16(),
         "gamma": r(64), "beta": r(64), "hx": r(300, 40).bfloat16(), "hw": r(700, 40).bfloat16(),
         "labels": torch.randint(-1, 700, (300,), generator=g, device="cuda"), "bx": r(900, 64).bfloat16(),
         "bw": r(3000, 64).bfloat16(), "bl": torch.randint(0, 3000, (900,), generator=g, device="cuda"),
         "g1": r(60, 200), "g2": r(2, 150, 260)}

    def run():
        out = []
        for x, dy, k, ga, be in ((d["x1"], d["dy1"], 8, d["gamma"], d["beta"]), (d["x2"], d["dy2"], 4, None, None)):
            stats = torch.empty((x.shape[0], k, 2), device="cuda")
            out.append(conv.group_norm(x, k, ga, be, act="mish", stats=stats))
            out += conv.group_norm_grad(dy, x, stats, ga, be, act="mish")
        out += conv.head_loss_grad(d["hx"], d["hw"], d["labels"])
        out += conv.head_loss_grad(d["bx"], d["bw"], d["bl"])
        out += conv.head_loss(d["hx"], d["hw"], d["labels"])
        out += [conv.orthogonalize(d["g1"]), conv.orthogonalize(d["g2"])]
        return out
    return d, run


def test_every_call_repeats_bit_for_bit():
    _, run = all_calls(1)
    first = [t.clone() for t in run()]
    for _ in range(3):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)


def test_graph_replays_match_eager():
    d, run = all_calls(2)
    run()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured = run()
    for seed in range(4):
        fresh, eager = all_calls(10 + seed)
        want = [t.clone() for t in eager()]  # eager work between the replays
        for k in d:
            d[k].copy_(fresh[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, captured):
            assert torch.equal(a, b), seed


def test_side_stream_and_given_scratch():
    d, run = all_calls(3)
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # an explicit stream, with outputs and scratch of the caller's
    y = torch.empty_like(d["x2"])
    ws = torch.empty(train.group_norm_ws_bytes(d["x2"], 4, act="mish"), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    torch.cuda.synchronize()
    conv.group_norm(d["x2"], 4, act="mish", y=y, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(y, conv.group_norm(d["x2"], 4, act="mish"))
    out = torch.empty_like(d["g2"], dtype=torch.bfloat16)
    ws = torch.full((train.orthogonalize_ws_bytes(2, 150, 260),), 255, dtype=torch.uint8, device="cuda")
    conv.orthogonalize(d["g2"], out=out, ws=ws)
    assert torch.equal(out, conv.orthogonalize(d["g2"]))
    ws = torch.full((train.head_loss_ws_bytes(300, 40, 700, grad=True),), 255, dtype=torch.uint8, device="cuda")
    a, b = conv.head_loss_grad(d["hx"], d["hw"], d["labels"], ws=ws), conv.head_loss_grad(d["hx"], d["hw"], d["labels"])
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_too_small_scratch_is_refused():
    x = torch.randn((1, 150, 150, 16), device="cuda")
    ws = torch.empty(64, dtype=torch.uint8, device="cuda")
    for call in (lambda: conv.group_norm(x, 4, ws=ws), lambda: conv.orthogonalize(x.view(150, -1), ws=ws),
                 lambda: conv.head_loss(torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda"),
                                        torch.zeros((5, 8), dtype=torch.bfloat16, device="cuda"),
                                        torch.zeros(4, dtype=torch.int64, device="cuda"), ws=ws)):
        with pytest.raises(conv.ConvError) as e:
            call()
        assert e.value.name == "CONV_E_SCRATCH"
    with pytest.raises(ValueError):
        conv.group_norm(x, 4, torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        conv.group_norm(x.transpose(1, 3), 4)
    with pytest.raises(ValueError):
        conv.head_loss(x.bfloat16(), torch.zeros((5, 16), dtype=torch.bfloat16, device="cuda"),
                       torch.zeros((1, 150, 149), dtype=torch.int64, device="cuda"))


def test_fitting_a_head_lowers_its_loss():
    """The operators together, on maps of a convolution layer: the loss starts
    at about the logarithm of the classes and falls by half."""
    from convolution_conv2d_nhwc_amd import fit
    losses = fit.run(steps=60, classes=50, quiet=True)
    assert abs(losses[0] - 3.912) < 0.5
    assert losses[-1] < 0.5 * losses[0], losses


# ------------------------------------------------------------ cases of one variant each --

@pytest.mark.parametrize("shape", [(1, 18, 25, 72, 1, "bf16"), (4, 15, 30, 576, 8, "bf16"), (1, 14, 15, 76, 4, "bf16"),
                                   (1, 11, 14, 104, 1, "f32"), (16, 17, 17, 448, 32, "f32"), (1, 3, 3, 301, 1, "f32"),
                                   (1, 3, 3, 301, 1, "bf16"), (1, 45, 10, 9, 3, "bf16")],
                         ids=lambda s: "x".join(map(str, s)))
def test_group_norm_of_1024_lanes_with_few_vectors(shape):
    """Maps of over 8 vectors for each of 512 lanes, but 3 or 4 for each of 1024."""
    n, h, w, c, groups, dtype = shape
    g = gen(c)
    x, dy = (torch.randn((n, h, w, c), generator=g).to(DT[dtype]) for _ in range(2))
    gamma, beta = 1 + 0.3 * torch.randn(c, generator=g), 0.3 * torch.randn(c, generator=g)
    check_norm(x, groups, gamma, beta, "silu", dtype, dy=dy)


def test_group_norm_refuses_a_broadcast_map():
    """One pixel's memory is not a map's: nothing is read past it."""
    x, dy = torch.ones((1, 1, 1, 64), device="cuda").expand(2, 8, 8, 64), torch.ones((2, 8, 8, 64), device="cuda")
    with pytest.raises(ValueError):
        conv.group_norm(x, 4)
    with pytest.raises(ValueError):
        train.group_norm_ws_bytes(x, 4)
    with pytest.raises(ValueError):
        conv.group_norm_grad(dy, x, torch.ones((2, 4, 2), device="cuda"))
    with pytest.raises(ValueError):
        conv.group_norm_grad(x, dy, torch.ones((2, 4, 2), device="cuda"))


@pytest.mark.parametrize("form", ["stream", "address"])
def test_memory_of_a_call_with_a_stream_is_that_streams(form, monkeypatch):
    """Outputs and scratch that the wrapper allocates belong to the stream that
    uses them, wherever the caller is; results are those of the current stream."""
    d, _ = all_calls(6)
    stats = torch.empty((1, 4, 2), device="cuda")
    calls = [lambda **k: conv.group_norm(d["x2"], 4, act="mish", stats=stats, **k),
             lambda **k: conv.group_norm_grad(d["dy2"], d["x2"], stats, act="mish", **k),
             lambda **k: conv.head_loss(d["bx"], d["bw"], d["bl"], **k),
             lambda **k: conv.head_loss_grad(d["bx"], d["bw"], d["bl"], **k),
             lambda **k: conv.orthogonalize(d["g2"], **k)]
    flat = lambda r: list(r) if isinstance(r, tuple) else [r]  # noqa: E731
    want = [[t.clone() for t in flat(c())] for c in calls]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = []
    for name in ("empty", "empty_like"):
        def spy(*a, _real=getattr(torch, name), **k):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return _real(*a, **k)
        monkeypatch.setattr(torch, name, spy)
    here = torch.cuda.current_stream()
    for call, ref in zip(calls, want):
        seen.clear()
        got = flat(call(stream=side if form == "stream" else side.cuda_stream))
        assert seen and set(seen) == {side.cuda_stream}
        assert torch.cuda.current_stream() == here
        side.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
