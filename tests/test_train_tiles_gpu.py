"""The training-side operators at the sizes that take each of their products'
tiles (tests/train_cases.py), against the formula in 64 bits."""
import pytest
import torch

import convolution_conv2d_nhwc_amd as conv
from convolution_conv2d_nhwc_amd import train
from tests import test_train_gpu as T
from tests.train_cases import LOSS_TILES, ORTHO_TILES

pytestmark = pytest.mark.gpu


def check_loss_by_blocks(x, w, labels, weights, monkeypatch):
    """As check_loss, with the reference on the device, a block of rows at a
    time; a sum's longest chain is that of its 32-wide products."""
    rows, (v, c) = x.shape[0], w.shape
    monkeypatch.setattr(T, "DEPTH", max(T.DEPTH, max(rows, v) // 32 + 64))
    got = T.run_loss(x, w, labels, weights)
    kept = (labels >= 0) & (labels < v)
    k = weights if weights is not None else torch.full((rows,), 1.0 / int(kept.sum()), device="cuda")
    total = torch.zeros(2, dtype=torch.float64, device="cuda")
    dw = torch.zeros((2, v, c), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // v)
    for i in range(0, rows, step):
        sl = slice(i, i + step)
        r = T.loss_ref(x[sl], w, labels[sl], k[sl])
        for name in ("loss", "dx"):
            ref, tol = r[name]
            bad = ~((got[name][sl].double() - ref).abs() <= tol)
            assert not bad.any(), (name, i, int(bad.sum()), bad.nonzero()[:4].tolist())
        total += torch.stack([t.cuda() for t in r["total"]])
        dw[0] += r["dw"][0]
        dw[1] += r["dw"][1]
    assert (got["total"].double() - total[0]).abs() <= total[1]
    # the blocks' tolerances hold half a step of each block's dw; the sum's may be larger
    bad = ~((got["dw"].double() - dw[0]).abs() <= dw[1] + T.HALF * dw[0].abs())
    assert not bad.any(), ("dw", int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("shape", LOSS_TILES, ids=lambda s: "x".join(map(str, s)))
def test_head_loss_tile(shape, monkeypatch):
    x, w, labels, g = T.loss_case(*shape)
    x[3::5] = float("nan")  # of rows left out: never used
    labels[3::5] = -100
    labels[4] = shape[2]    # one past the last class
    weights = torch.rand(shape[0], generator=g, device="cuda") / shape[0] if shape[0] % 2 else None
    check_loss_by_blocks(x, w, labels, weights, monkeypatch)


def ortho_ref(g, steps=5, coeffs=train.MUON_COEFFS, eps=1e-7):
    """As test_train_gpu's, a matrix at a time, on g's device."""
    a, b, c = coeffs
    out = []
    for m in g.double():
        x = (m if m.shape[0] <= m.shape[1] else m.t()).contiguous()
        x = x / (x.norm() + eps)
        for _ in range(steps):
            p = x @ x.t().contiguous()
            x = a * x + (b * p + c * (p @ p)) @ x
        out.append(x if m.shape[0] <= m.shape[1] else x.t())
    return torch.stack(out)


def check_entries(got, ref):
    """Every entry: half a step of the bf16 store, and what the products leave.
    Their operands are off by up to 2^-11 of themselves; in quadrature over five
    steps of three products 2^-9 of an entry's mean size, four times that at most."""
    rms = ref.flatten(-2).norm(dim=-1)[:, None, None] / (ref.shape[-1] * ref.shape[-2]) ** 0.5
    t = 2.0 ** -7 * rms
    bad = ~((got.double() - ref).abs() <= T.HALF * (ref.abs() + t) + t)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


def ortho_case(shape, dtype, seed=0):
    b, m, n = shape
    g = torch.Generator(device="cuda").manual_seed(m + n + seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    r = max(1, min(m, n) // 8)
    low = torch.stack([randn(m, r) @ randn(r, n) for _ in range(b)])
    return (1e-3 * (randn(b, m, n) + low)).to(T.DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", ORTHO_TILES, ids=lambda s: "x".join(map(str, s)))
def test_orthogonalize_tile(shape, dtype):
    x = ortho_case(shape, dtype)
    off = 1 if dtype == "bf16" else 0  # out aligned to its elements only
    out = torch.full((x.numel() + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
    conv.orthogonalize(x, out=out[off:off + x.numel()].view(shape))
    check_entries(out[off:off + x.numel()].view(shape), ortho_ref(x))
    assert torch.isnan(out[:off]).all() and torch.isnan(out[off + x.numel():]).all()
