"""Sizes at which the training-side operators take each of their kernels, shared
by the tests that run them on the GPU and by the CPU test that holds the sizes to
the kernels they are there for."""
import ctypes

from convolution_conv2d_nhwc_amd import train

# rows, channels, classes: every tile of every product of the head loss, at sizes
# that are no multiple of a tile
LOSS_TILES = [
    (66, 67, 8283), (7234, 260, 1603), (1557, 652, 71), (41, 132, 18166), (6923, 533, 71), (41, 132, 33793),
    (2241, 68, 17538), (6353, 134, 5479), (6841, 130, 5113), (8343, 899, 1115), (3301, 515, 20011),
    (1367, 38, 75), (44, 65, 18449), (3783, 65, 3079), (2979, 66, 3798),
    (3301, 520, 20011),   # read in place
    (6401, 264, 45007),   # 256 tiles in pieces of the classes
]

# batch, rows, columns: every tile of the update's products
ORTHO_TILES = [
    (2, 65, 70), (16, 389, 388), (16, 641, 665), (16, 1097, 1026), (2, 2050, 333), (16, 70, 2819), (16, 321, 326),
    (1, 1990, 2050), (1, 1000, 4600), (1, 4600, 1000), (6, 1333, 1409),
]


def fields(text):
    """The key=value fields of a describe entry point's text."""
    return {k: int(v) if v.isdigit() else v for k, v in (f.split("=") for f in text.split() if "=" in f)}


def described(call, *args):
    buf = ctypes.create_string_buffer(512)
    assert call(*args, buf, 512) == 0
    return fields(buf.value.decode())


def loss_kernels(rows, c, classes):
    """The kernels that head_loss_grad takes: (product, tile x workgroups a CU
    [, whether it writes partial sums])."""
    f = described(train._L().conv_head_loss_describe, train._HeadDesc(rows, c, classes, 1, 8), 1, 16)
    got = {("logits", f["logits"]), ("g", f["g"])}
    if f["pair"]:
        got.add(("pair",))
    else:
        got |= {("dx", f["dx"], f["dx_part"]), ("dw", f["dw"], f["dw_part"])}
    if f["pieces"] > 1:
        got.add(("pieces", f["g"]))
    return got


def ortho_kernels(batch, rows, cols):
    f = described(train._L().conv_orthogonalize_describe, train._OrthoDesc(batch, rows, cols, 0, 5, 1.0, 0.0, 0.0, 0.0))
    return {("sym", f["sym"]), ("step", f["step"])} if "sym" in f else {("small", f["blocks"])}
