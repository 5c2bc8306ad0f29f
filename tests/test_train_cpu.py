"""The training-side operators' boundary, on the CPU: every malformed call is
refused with its named error before anything would be enqueued (the addresses
are made up and never read), and the scratch sizes are consistent."""
import ctypes
import os

import pytest
import torch

from convolution_conv2d_nhwc_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.library_path()), reason="libconv_nhwc.so not built")

if os.path.exists(_lib.library_path()):
    from convolution_conv2d_nhwc_amd import train
    from tests.train_cases import LOSS_TILES, ORTHO_TILES, described, loss_kernels, ortho_kernels

E_NULL, E_SHAPE, E_UNSUPPORTED, E_ALIGN, E_ALIAS, E_SCRATCH = -1, -2, -3, -4, -5, -8
A = [(i + 1) << 36 for i in range(12)]  # addresses far apart
BIG = 1 << 40


def norm_desc(**kw):
    d = dict(n=2, h=4, w=4, c=16, x_pixel_stride=0, groups=4, dtype=1, act=0, eps=1e-5)
    d.update(kw)
    return train._NormDesc(**d)


def head_desc(**kw):
    d = dict(rows=10, c=16, classes=30, dtype=1, label_bytes=8)
    d.update(kw)
    return train._HeadDesc(**d)


def ortho_desc(**kw):
    d = dict(batch=1, rows=100, cols=200, dtype=0, steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7)
    d.update(kw)
    return train._OrthoDesc(**d)


def norm(d, p, ws=BIG):
    return train._L().conv_group_norm(d, *p[:6], ws, None)


def norm_grad(d, p, ws=BIG):
    return train._L().conv_group_norm_grad(d, *p[:9], ws, None)


NORM_BAD = [
    (dict(n=0), E_SHAPE), (dict(h=-1), E_SHAPE), (dict(w=0), E_SHAPE), (dict(c=0), E_SHAPE), (dict(groups=0), E_SHAPE),
    (dict(groups=3), E_SHAPE), (dict(x_pixel_stride=15), E_SHAPE), (dict(x_pixel_stride=-1), E_SHAPE),
    (dict(eps=-1.0), E_SHAPE), (dict(eps=float("nan")), E_SHAPE), (dict(eps=float("inf")), E_SHAPE),
    (dict(dtype=2), E_UNSUPPORTED), (dict(dtype=-1), E_UNSUPPORTED), (dict(act=5), E_UNSUPPORTED),
    (dict(act=-1), E_UNSUPPORTED), (dict(n=65536), E_UNSUPPORTED), (dict(c=65536 * 4), E_UNSUPPORTED),
    (dict(h=1 << 20, w=1 << 20), E_UNSUPPORTED), (dict(h=1 << 62, w=1 << 62), E_UNSUPPORTED),
    (dict(n=16, h=4096, w=1024, c=16, x_pixel_stride=32), E_UNSUPPORTED),  # x of 2^32 bytes
]


@pytest.mark.parametrize("kw,code", NORM_BAD)
def test_group_norm_refuses_descriptions(kw, code):
    d = norm_desc(**kw)
    assert norm(d, A) == code
    assert norm_grad(d, A) == code
    for grad in (0, 1):
        assert train._L().conv_group_norm_ws_bytes(d, grad) == code


def swap(p, i, v):
    p = list(p)
    p[i] = v
    return p


def test_group_norm_refuses_pointers():
    d = norm_desc()
    # x, gamma, beta, y, stats, ws
    assert train._L().conv_group_norm(None, *A[:6], BIG, None) == E_NULL
    for i in (0, 3):
        assert norm(d, swap(A, i, None)) == E_NULL
    assert norm(d, swap(A, 0, A[0] + 1)) == E_ALIGN
    assert norm(norm_desc(dtype=0), swap(A, 3, A[3] + 2)) == E_ALIGN
    assert norm(d, swap(A, 1, A[1] + 2)) == E_ALIGN
    assert norm(d, swap(A, 5, A[5] + 64)) == E_ALIGN
    assert norm(d, swap(A, 3, A[0] + 64)) == E_ALIAS  # y inside x
    assert norm(d, swap(A, 4, A[3])) == E_ALIAS       # stats on y
    assert norm(d, swap(A, 4, A[1])) == E_ALIAS       # stats on gamma
    wide = norm_desc(n=1, h=500, w=500, c=64, groups=4)
    need = train._L().conv_group_norm_ws_bytes(wide, 0)
    assert need > 0
    assert norm(wide, swap(A, 5, None)) == E_NULL
    assert norm(wide, A, 8) == E_SCRATCH
    assert norm(wide, swap(A, 5, A[0] + 256)) == E_ALIAS
    # x, dy, stats, gamma, beta, dx, dgamma, dbeta, ws
    assert train._L().conv_group_norm_grad(None, *A[:9], BIG, None) == E_NULL
    for i in (0, 1, 2, 5):
        assert norm_grad(d, swap(A, i, None)) == E_NULL
    assert norm_grad(d, swap(A, 1, A[1] + 1)) == E_ALIGN
    assert norm_grad(d, swap(A, 2, A[2] + 1)) == E_ALIGN
    assert norm_grad(d, swap(A, 8, A[8] + 16)) == E_ALIGN
    assert norm_grad(d, swap(A, 5, A[1])) == E_ALIAS  # dx on dy
    assert norm_grad(d, swap(A, 7, A[6])) == E_ALIAS  # dbeta on dgamma
    assert norm_grad(d, A, 8) == E_SCRATCH            # two images: sums of channels
    assert norm_grad(d, swap(A, 8, None)) == E_NULL


def head(d, p, grad, ws=BIG):
    L = train._L()
    return L.conv_head_loss_grad(d, *p[:9], ws, None) if grad else L.conv_head_loss(d, *p[:7], ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), E_SHAPE), (dict(c=0), E_SHAPE), (dict(classes=-5), E_SHAPE), (dict(dtype=0), E_UNSUPPORTED),
    (dict(label_bytes=2), E_UNSUPPORTED), (dict(c=65537), E_UNSUPPORTED), (dict(rows=1 << 22), E_UNSUPPORTED),
    (dict(classes=1 << 22), E_UNSUPPORTED), (dict(rows=1 << 20, c=2048), E_UNSUPPORTED),
    (dict(classes=1 << 62), E_UNSUPPORTED),
])
def test_head_loss_refuses_descriptions(kw, code):
    d = head_desc(**kw)
    for grad in (0, 1):
        assert head(d, A, grad) == code
        assert train._L().conv_head_loss_ws_bytes(d, grad) == code


def test_head_loss_refuses_pointers():
    d = head_desc()
    assert head(None, A, 0) == E_NULL and head(None, A, 1) == E_NULL
    # x, w, labels, weights, loss, total, [dx, dw,] ws
    for i in (0, 1, 2, 4, 5, 6):
        assert head(d, swap(A, i, None), 0) == E_NULL
    for i in (6, 7, 8):
        assert head(d, swap(A, i, None), 1) == E_NULL
    assert head(d, swap(A, 0, A[0] + 1), 0) == E_ALIGN
    assert head(d, swap(A, 2, A[2] + 4), 0) == E_ALIGN
    assert head(head_desc(label_bytes=4), swap(A, 2, A[2] + 2), 0) == E_ALIGN
    assert head(d, swap(A, 3, A[3] + 2), 0) == E_ALIGN
    assert head(d, swap(A, 7, A[7] + 1), 1) == E_ALIGN
    assert head(d, swap(A, 8, A[8] + 128), 1) == E_ALIGN
    assert head(d, A, 0, 100) == E_SCRATCH
    assert head(d, A, 1, train._L().conv_head_loss_ws_bytes(head_desc(), 0)) == E_SCRATCH
    assert head(d, swap(A, 4, A[3]), 0) == E_ALIAS  # loss on weights
    assert head(d, swap(A, 6, A[0]), 1) == E_ALIAS  # dx on x
    assert head(d, swap(A, 7, A[6] + 32), 1) == E_ALIAS


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), E_SHAPE), (dict(rows=0), E_SHAPE), (dict(cols=-1), E_SHAPE), (dict(steps=0), E_SHAPE),
    (dict(steps=101), E_SHAPE), (dict(a=float("nan")), E_SHAPE), (dict(c=float("inf")), E_SHAPE),
    (dict(eps=-1e-9), E_SHAPE), (dict(dtype=2), E_UNSUPPORTED), (dict(batch=65536), E_UNSUPPORTED),
    (dict(rows=32769), E_UNSUPPORTED), (dict(rows=32768, cols=32768), E_UNSUPPORTED),
    (dict(batch=60000, rows=1000, cols=1000), E_UNSUPPORTED),
])
def test_orthogonalize_refuses_descriptions(kw, code):
    d = ortho_desc(**kw)
    assert train._L().conv_orthogonalize(d, *A[:3], BIG, None) == code
    assert train._L().conv_orthogonalize_ws_bytes(d) == code


def test_orthogonalize_refuses_pointers():
    L, d = train._L(), ortho_desc()
    assert L.conv_orthogonalize(None, *A[:3], BIG, None) == E_NULL
    for i in range(3):
        assert L.conv_orthogonalize(d, *swap(A, i, None)[:3], BIG, None) == E_NULL
    assert L.conv_orthogonalize(d, *swap(A, 0, A[0] + 2)[:3], BIG, None) == E_ALIGN
    assert L.conv_orthogonalize(d, *swap(A, 2, A[2] + 4)[:3], BIG, None) == E_ALIGN
    assert L.conv_orthogonalize(d, *A[:3], 1000, None) == E_SCRATCH
    assert L.conv_orthogonalize(d, *swap(A, 1, A[0] + 400)[:3], BIG, None) == E_ALIAS
    # a matrix that fits one workgroup needs no scratch, and still checks the rest
    small = ortho_desc(rows=64, cols=576)
    assert L.conv_orthogonalize_ws_bytes(small) == 0
    assert L.conv_orthogonalize(small, A[0], A[0], None, 0, None) == E_ALIAS


def test_scratch_sizes():
    L = train._L()
    assert L.conv_group_norm_ws_bytes(norm_desc(n=1, h=20, w=20, c=512, groups=32), 0) == 0  # one launch
    assert L.conv_group_norm_ws_bytes(norm_desc(n=1, h=20, w=20, c=512, groups=32), 1) == 0
    # pieces of g bound the gradient's scratch: 512 MiB of g at most, besides partial sums and copies
    rows, classes, c = 100000, 100000, 64
    need = L.conv_head_loss_ws_bytes(head_desc(rows=rows, c=c, classes=classes), 1)
    fwd = L.conv_head_loss_ws_bytes(head_desc(rows=rows, c=c, classes=classes), 0)
    assert need - fwd < (512 << 20) + 17 * 4 * rows * c + 4 * (rows + classes) * c + (1 << 20)
    assert rows * classes * 2 > 10 * (need - fwd)


@pytest.mark.parametrize("call", [
    lambda t: t.group_norm(torch.zeros(1, 4, 4, 8), 2),
    lambda t: t.group_norm_grad(torch.zeros(1, 4, 4, 8), torch.zeros(1, 4, 4, 8), torch.zeros(1, 2, 2)),
    lambda t: t.head_loss(torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16),
                          torch.zeros(4, dtype=torch.int64)),
    lambda t: t.head_loss(torch.zeros(4, 8), torch.zeros(5, 9), torch.zeros(4, dtype=torch.int64)),
    lambda t: t.orthogonalize(torch.zeros(4, 8)),
    lambda t: t.orthogonalize(torch.zeros(8)),
    lambda t: t.orthogonalize(torch.zeros(8, 8, dtype=torch.float16)),
])
def test_python_refuses_host_tensors_and_shapes(call):
    with pytest.raises(ValueError):
        call(train)


def test_ws_bytes_from_python_raise_named_errors():
    with pytest.raises(_lib.ConvError) as e:
        train.head_loss_ws_bytes(0, 8, 8)
    assert e.value.name == "CONV_E_SHAPE"
    with pytest.raises(_lib.ConvError) as e:
        train.orthogonalize_ws_bytes(1, 40000, 10)
    assert e.value.name == "CONV_E_UNSUPPORTED"
    assert train.head_loss_ws_bytes(100, 64, 1000, grad=True) > train.head_loss_ws_bytes(100, 64, 1000) > 0


# n, h, w, c, groups, dtype: maps whose tile needs 3 or 4 vectors of 1024 lanes but over 8 of 512
ODD_LANES = [(1, 18, 25, 72, 1, 1), (4, 15, 30, 576, 8, 1), (1, 14, 15, 76, 4, 1), (1, 11, 14, 104, 1, 0),
             (16, 17, 17, 448, 32, 0), (1, 3, 3, 301, 1, 0)]


def norm_plan_problem(shape, dtype, align, grad):
    n, h, w, c, groups = shape
    p = described(train._L().conv_group_norm_describe, norm_desc(n=n, h=h, w=w, c=c, groups=groups, dtype=dtype), grad, align)
    # the kernels are built for 512 lanes, and for 1024 with 8 vectors each
    if p["threads"] not in (512, 1024) or (p["threads"] == 1024 and p["r"] != 8):
        return "lanes"
    if p["r"] not in (0, 1, 2, 4, 8) or p["ct"] % p["vec"] or p["ct"] > 512:
        return "variant"
    if p["ppi"] < 1 or p["ppi"] * (p["ct"] // p["vec"]) > p["threads"]:
        return "more lanes than launched"
    cg = c // groups
    covered = p["ctiles"] // p["tpg"] * p["gpt"] >= groups and (p["gpt"] * cg == p["ct"] if p["tpg"] == 1 else p["tpg"] * p["ct"] >= cg)
    if not covered or c % p["vec"]:
        return "channels left over"
    if p["r"] and p["r"] * p["ppi"] < h * w:
        return "pixels left over"
    if p["chunks"] * p["cpix"] < h * w or (p["chunks"] - 1) * p["cpix"] >= h * w:
        return "chunks"
    return None


@pytest.mark.parametrize("grad", [0, 1])
@pytest.mark.parametrize("shape", ODD_LANES, ids=lambda s: "x".join(map(str, s)))
def test_group_norm_plan_of_1024_lanes(shape, grad):
    for align in (2, 4, 8, 16):
        assert norm_plan_problem(shape[:5], shape[5], align, grad) is None


@pytest.mark.parametrize("dtype", [0, 1])
def test_group_norm_plan_covers_the_map(dtype):
    """Every plan's lanes exist, and reach every channel and pixel."""
    for cg in list(range(1, 130)) + [144, 171, 192, 256, 301, 341, 400, 511, 512, 513, 640, 1030]:
        for groups in (1, 2, 3, 8, 32):
            if cg * groups > 4096:
                continue
            for hw in list(range(1, 70, 3)) + [100, 150, 289, 450, 777, 1600, 6400, 22500]:
                for n, grad, align in ((1, 0, 16), (4, 1, 16), (1, 1, 2)):
                    shape = (n, 1, hw, cg * groups, groups)
                    assert norm_plan_problem(shape, dtype, align, grad) is None, (shape, grad, align)


@pytest.mark.parametrize("x", [
    torch.zeros(1, 1, 1, 64).expand(2, 8, 8, 64),         # one pixel for the whole map
    torch.zeros(2, 1, 1, 64).expand(2, 8, 8, 64),
    torch.zeros(2, 8, 1, 64).expand(2, 8, 8, 64),
    torch.zeros(1, 8, 8, 64).expand(2, 8, 8, 64),
    torch.zeros(1, 1, 1, 1).expand(2, 8, 8, 1),
    torch.zeros(2, 8, 8, 1).expand(2, 8, 8, 64),
    torch.zeros(4096).as_strided((1, 4, 4, 64), (512, 128, 32, 1)),  # pixels that overlap
    torch.zeros(2, 64, 8, 8).permute(0, 2, 3, 1),
    torch.zeros(2, 8, 16, 64)[:, :, :8],
], ids=lambda t: "%s-%s" % ("x".join(map(str, t.shape)), "x".join(map(str, t.stride()))))
def test_maps_whose_pixels_do_not_follow_each_other_are_refused(x):
    with pytest.raises(ValueError):
        train._pixel_pitch(x)


@pytest.mark.parametrize("x,pitch", [
    (torch.zeros(2, 8, 8, 64), 64), (torch.zeros(2, 8, 8, 100)[..., 20:84], 100), (torch.zeros(2, 8, 8, 5)[..., 2:3], 5),
    (torch.zeros(2, 8, 16, 64)[:, :, ::2], 128),  # every other pixel is one step
    (torch.zeros(1, 1, 1, 64).expand(1, 1, 1, 64), 64), (torch.zeros(1, 1, 4, 100)[..., :64], 100),
    (torch.zeros(1, 4, 1, 100)[..., :64], 100), (torch.zeros(4, 1, 1, 100)[..., :64], 100),
    (torch.zeros(1, 1, 1, 100)[..., :64], 64), (torch.zeros(64).as_strided((1, 1, 1, 64), (0, 0, 0, 1)), 64),
])
def test_pixel_pitch_of_maps_and_slices(x, pitch):
    assert (train._pixel_pitch(x) or x.shape[3]) == pitch


class FakeMap:
    """What _norm_of looks at of a device map."""
    shape, dtype, is_cuda = (2, 4, 4, 16), torch.float32, True

    def dim(self):
        return 4

    def is_contiguous(self):
        return True


def test_arguments_changed_in_place_are_read_again():
    eps, steps, a = torch.tensor(0.25), torch.tensor(5), torch.tensor(2.0)
    assert train._norm_of(FakeMap(), 4, eps, "none", False)[0].eps == 0.25
    d = train._ortho_of(1, 100, 200, torch.float32, steps, a, 0.0, 0.0, eps)[0]
    assert (d.steps, d.a, d.eps) == (5, 2.0, 0.25)
    eps.fill_(0.5), steps.fill_(2), a.fill_(3.0)
    assert train._norm_of(FakeMap(), 4, eps, "none", False)[0].eps == 0.5
    d = train._ortho_of(1, 100, 200, torch.float32, steps, a, 0.0, 0.0, eps)[0]
    assert (d.steps, d.a, d.eps) == (2, 3.0, 0.5)


def test_sizes_are_whole_numbers_whatever_was_asked_before():
    train._norm_of(FakeMap(), 4, 1e-5, "none", False)
    with pytest.raises(TypeError):
        train._norm_of(FakeMap(), 4.0, 1e-5, "none", False)
    train._ortho_of(1, 100, 200, torch.float32, 5, 1.0, 0.0, 0.0, 1e-7)
    with pytest.raises(TypeError):
        train._ortho_of(1, 100, 200, torch.float32, 5.0, 1.0, 0.0, 0.0, 1e-7)


@pytest.mark.parametrize("call", [
    lambda t, s: t.group_norm(torch.zeros(1, 4, 4, 8), 2, stream=s),
    lambda t, s: t.group_norm_grad(torch.zeros(1, 4, 4, 8), torch.zeros(1, 4, 4, 8), torch.zeros(1, 2, 2), stream=s),
    lambda t, s: t.head_loss(torch.zeros(4, 8), torch.zeros(5, 8), torch.zeros(4, dtype=torch.int64), stream=s),
    lambda t, s: t.head_loss_grad(torch.zeros(4, 8), torch.zeros(5, 8), torch.zeros(4, dtype=torch.int64), stream=s),
    lambda t, s: t.orthogonalize(torch.zeros(4, 8), stream=s),
])
def test_host_tensors_are_refused_with_a_stream_too(call):
    with pytest.raises(ValueError):
        call(train, 1 << 40)


@pytest.mark.parametrize("rows,classes,c,ok", [
    (1 << 20, 1 << 18, 8, False), ((1 << 20) - 128, 1 << 18, 8, True), (1 << 18, 1 << 20, 200, False),
    (1 << 20, 1 << 18, 264, True), (1 << 21, 1 << 19, 264, False), ((1 << 21) - 256, 1 << 19, 264, True),
    ((1 << 22) - 64, (1 << 22) - 64, 8, False),
])
def test_head_loss_refuses_more_workgroups_than_a_launch_has(rows, classes, c, ok):
    """256 lanes a workgroup, fewer than 2^32 a launch: refused by name, not by
    the launch after others are already enqueued."""
    d = head_desc(rows=rows, classes=classes, c=c)
    for grad in (0, 1):
        need = train._L().conv_head_loss_ws_bytes(d, grad)
        assert need > 0 if ok else need == E_UNSUPPORTED
        if not ok:
            assert head(d, A, grad) == E_UNSUPPORTED


TILES = ["64x1", "64x2", "128x1", "128x2", "256x1"]  # side x workgroups a CU


def test_every_product_of_the_head_loss_has_a_case():
    """The GPU tests' sizes reach each kernel that the rules can choose."""
    got = set().union(*(loss_kernels(*s) for s in LOSS_TILES + [(125, 64, 1000)]))
    want = {(p, t) for p in ("logits", "g") for t in TILES}
    want |= {(p, t, part) for p in ("dx", "dw") for t in TILES for part in (0, 1)}
    want |= {("pair",), ("pieces", "256x1")}
    assert not want - got, sorted(want - got)


def test_every_product_of_the_update_has_a_case():
    small = [(1, 64, n) for n in (256, 512, 768, 1024)]
    got = set().union(*(ortho_kernels(*s) for s in ORTHO_TILES + small))
    want = {(p, t) for p in ("sym", "step") for t in TILES} | {("small", b) for b in (1, 2, 3, 4)}
    assert not want - got, sorted(want - got)


def test_describe_refuses_as_the_calls_do():
    L, buf = train._L(), ctypes.create_string_buffer(512)
    for call, good, bad in ((lambda *a: L.conv_group_norm_describe(a[0], 0, 16, *a[1:]), norm_desc(), norm_desc(c=0)),
                            (lambda *a: L.conv_head_loss_describe(a[0], 1, 16, *a[1:]), head_desc(), head_desc(c=0)),
                            (L.conv_orthogonalize_describe, ortho_desc(), ortho_desc(rows=0))):
        assert call(None, buf, 512) == E_NULL and call(good, None, 512) == E_NULL and call(good, buf, 0) == E_NULL
        assert call(bad, buf, 512) == E_SHAPE
        assert call(good, buf, 8) == 0 and len(buf.value) == 7  # cut to the buffer
