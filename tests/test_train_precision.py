"""What the update and the head loss's gradients lose besides the bf16 rounding of
their results, against the arithmetic that include/conv_train.h describes.

The kernels' roundings are emulated in elementary operations (the oracle here),
and the error that these leave before the last rounding is compared with the
kernels'. Rounding is monotone and keeps differences on average, E |rd(a) - rd(b)|
= E |a - b| for errors below a step, so the mean of |rd(result) - rd(reference)|
measures the error under the last rounding, which the result's own rounding would
otherwise hide. The CPU tests plant in the emulation what the kernels keep apart
(the second fp16 of X, the diagonals, the label's remainder) and show that each
loss leaves the bounds that the GPU tests hold the kernels to.
"""
import pytest
import torch

import convolution_conv2d_nhwc_amd as conv
from convolution_conv2d_nhwc_amd import train


def rd(t):
    return t.float().bfloat16().double()


# ------------------------------------------------------------ orthogonalisation --

def ortho_exact(g, steps=5, coeffs=train.MUON_COEFFS):
    a, b, c = coeffs
    x = g.double() / (g.double().norm() + 1e-7)
    for _ in range(steps):
        p = x @ x.t().contiguous()
        x = a * x + (b * p + c * (p @ p)) @ x
    return x


def ortho_emulated(g, steps=5, coeffs=train.MUON_COEFFS, pair=True, diag_a=True, diag_q=True):
    """The wide g's update with fp16 operands: X as a pair, A and Q as a diagonal
    in 32 bits and fp16 beside it, scaled as in the kernels."""
    a, b, c = coeffs
    sx, so, sr = 256.0, 4096.0, 1024.0
    half = lambda t: t.half().float()  # noqa: E731
    y = (g.double() / (g.double().norm() + 1e-7)).float() * sx
    for _ in range(steps):
        hi = half(y)
        lo = half(y - hi) if pair else torch.zeros_like(hi)
        gram = (hi @ hi.t().contiguous()) / (sx * sx)
        d = gram.diagonal().clone() if diag_a else torch.zeros_like(gram[0])
        o = half((gram - torch.diag(d)) * so) / so
        q = b * (o + torch.diag(d)) + c * (o @ o + (d[:, None] + d[None, :]) * o + torch.diag(d * d))
        q += a * torch.eye(len(q), device=q.device)
        e = q.diagonal().clone() if diag_q else torch.zeros_like(q[0])
        r = half((q - torch.diag(e)) * sr) / sr
        y = e[:, None] * (hi + lo) + r @ hi
    return y / sx


def ortho_gradient(m, n, device="cpu"):
    g = torch.Generator(device=device).manual_seed(m + n)
    r = max(1, min(m, n) // 8)
    randn = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    return 1e-3 * (randn(m, n) + randn(m, r) @ randn(r, n))


def ortho_excess(got, g):
    """(the mean error under the last rounding over the emulation's, its bound).
    Two orders of the sums give two samples of the same roundings: about one entry
    in twelve falls on another side, and 12 / sqrt(N) are over three standard
    deviations of that count; a tenth more for what a row's entries share."""
    exact = ortho_exact(g)
    mean = (ortho_emulated(g).double() - exact).abs().mean()
    return float((rd(got) - rd(exact)).abs().mean() / mean), 1.1 + 12 / g.numel() ** 0.5


@pytest.mark.parametrize("m,n", [(33, 100), (64, 576), (129, 513), (250, 700)])
def test_order_of_the_sums_does_not_matter_to_the_update(m, n):
    g = ortho_gradient(m, n)
    gen = torch.Generator().manual_seed(1)
    p, q = torch.randperm(m, generator=gen), torch.randperm(n, generator=gen)
    other = torch.empty_like(g)
    other[p[:, None], q[None, :]] = ortho_emulated(g[p][:, q].contiguous())
    excess, bound = ortho_excess(other, g)
    assert excess <= bound, (excess, bound)


@pytest.mark.parametrize("loss", ["pair", "diag_a", "diag_q"])
@pytest.mark.parametrize("m,n", [(64, 576), (129, 513), (250, 700)])  # the bound's 12 / sqrt(N) is below 1 / 16 here
def test_planted_losses_of_the_update_show(m, n, loss):
    g = ortho_gradient(m, n)
    excess, bound = ortho_excess(ortho_emulated(g, **{loss: False}), g)
    assert excess > bound, (excess, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(33, 100), (64, 576), (63, 1023), (64, 1024), (65, 70), (129, 513), (300, 300), (250, 1000),
                                 (700, 900), (388, 389), (70, 2819), (1000, 4600), (1990, 2050)])
def test_update_loses_what_its_operands_round(m, n, dtype):
    g = ortho_gradient(m, n, "cuda").to(dtype)
    excess, bound = ortho_excess(conv.orthogonalize(g), g)
    assert excess <= bound, (excess, bound)
    tall = conv.orthogonalize(g.t().contiguous()).t()
    excess, bound = ortho_excess(tall, g)
    assert excess <= bound, (excess, bound)


# ------------------------------------------------------------- head loss gradients --

def loss_gradients(x, w, labels, weights, rounded=True, remainder=True, logits=torch.float64):
    """(dx, dw) in 64 bits; rounded: with g in bf16, the label's remainder added
    back in 32 bits to dx and as bf16 to dw."""
    kept = (labels >= 0) & (labels < w.shape[0])
    at, r = torch.where(kept, labels, 0), torch.arange(len(labels), device=x.device)
    xd, wd = torch.where(kept[:, None], x.double(), 0.0), w.double()
    k = torch.where(kept, weights.double(), 0.0)
    g = torch.softmax(xd.to(logits) @ wd.to(logits).t().contiguous(), 1).double()
    g[r, at] -= 1.0
    g *= k[:, None]
    if not rounded:
        return g @ wd, g.t().contiguous() @ xd
    gb = rd(g)
    left = (g[r, at] - gb[r, at])[:, None]
    dx, dw = gb @ wd, gb.t().contiguous() @ xd
    if remainder:
        dx, dw = dx + left * wd[at], dw.index_add(0, at, rd(left) * xd)
    return dx, dw


def loss_inputs(rows, c, classes, device="cpu"):
    g = torch.Generator(device=device).manual_seed(rows + c)
    randn = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    w = randn(classes, c) * (2.0 / c ** 0.5)
    labels = torch.randint(0, classes, (rows,), generator=g, device=device)
    x = randn(rows, c) + w[labels]
    labels[::7] = -100
    weights = (torch.rand(rows, generator=g, device=device) + 0.5) / rows
    return x.bfloat16(), w.bfloat16(), labels, weights


def loss_difference(got, args):
    """For dx and dw: the mean of |rd(got) - rd(emulated)| over the emulation's own
    mean error. The logits' error (some 2^-20 of g) moves g's rounding of less than
    one entry in a hundred to the other side, and the results' of fewer."""
    exact, emulated = loss_gradients(*args, rounded=False), loss_gradients(*args)
    return [float((rd(a) - rd(b)).abs().mean() / (b - e).abs().mean()) for a, b, e in zip(got, emulated, exact)]


@pytest.mark.parametrize("shape", [(125, 64, 1000), (50, 32, 90), (700, 100, 1100), (66, 67, 4000), (1557, 200, 71)])
def test_planted_losses_of_the_gradients_show(shape):
    args = loss_inputs(*shape)
    assert max(loss_difference(loss_gradients(*args, logits=torch.float32), args)) <= 0.25
    assert min(loss_difference(loss_gradients(*args, remainder=False), args)) > 0.25


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(125, 64, 1000), (50, 32, 90), (700, 100, 1100), (66, 67, 8283), (1557, 652, 71),
                                   (2000, 24, 1030), (7234, 260, 1603), (6353, 134, 5479), (3301, 515, 8011)])
def test_gradients_lose_what_g_rounds(shape):
    args = loss_inputs(*shape, device="cuda")
    _, _, dx, dw = conv.head_loss_grad(*args)
    assert max(loss_difference((dx, dw), args)) <= 0.25
