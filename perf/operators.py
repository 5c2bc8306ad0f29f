"""The training-side operators next to the convolutions, as cases to measure.

Fitting a head on the maps that a convolution stack produces takes three
operators after the convolutions: group norm with its activation over NHWC
maps (forward and gradients), the softmax cross entropy of a 1x1 head over a
large set of classes with its gradients, and the orthogonalised update of a
weight matrix. ``own`` selects between their plain form in elementary torch
operations and the library's kernels.
"""
import math

import torch

own = False

NS_STEPS = 5
NS_COEFFS = (3.4445, -4.7750, 2.0315)


def listed():
    return [
        # one image's 20x20x512 map between two layers: latency counts
        {"name": "norm_20sq_512", "op": "norm", "n": 1, "h": 20, "w": 20, "c": 512, "groups": 32, "pitch": 512,
         "act": "silu", "dtype": "bf16"},
        # the batch-16 160x160x128 map of the neck sweep: the bandwidth-bound one
        {"name": "norm_160sq_128", "op": "norm", "n": 16, "h": 160, "w": 160, "c": 128, "groups": 32, "pitch": 128,
         "act": "mish", "dtype": "bf16"},
        # a channel slice of a joined map in float32, odd map size, 10 channels a group
        {"name": "norm_slice_f32", "op": "norm", "n": 3, "h": 41, "w": 39, "c": 60, "groups": 6, "pitch": 100,
         "act": "relu", "dtype": "f32"},
        # training step at the batch-16 40x40x512 map: forward, then all gradients
        {"name": "norm_train_40sq_512", "op": "norm_train", "n": 16, "h": 40, "w": 40, "c": 512, "groups": 32,
         "pitch": 512, "act": "silu", "dtype": "bf16"},
        # the same in float32 with odd sizes (9 groups of 10 channels)
        {"name": "norm_train_odd_f32", "op": "norm_train", "n": 2, "h": 77, "w": 53, "c": 90, "groups": 9,
         "pitch": 90, "act": "mish", "dtype": "f32"},
        # validation of a 1000-class head over one image's 20x20x1024 map
        {"name": "loss_400_1024_1000", "op": "loss", "rows": 400, "c": 1024, "classes": 1000, "ignored": 0.0,
         "weighted": False},
        # training of a small head on a 25x5x64 keyword map: latency counts
        {"name": "loss_train_125_64_1000", "op": "loss_train", "rows": 125, "c": 64, "classes": 1000,
         "ignored": 0.0, "weighted": False},
        # ragged: a 39x39 map, channels no multiple of 8, a prime class count, a quarter of the pixels unlabelled
        {"name": "loss_train_1521_250_10007", "op": "loss_train", "rows": 1521, "c": 250, "classes": 10007,
         "ignored": 0.25, "weighted": True},
        # a batch of 16 20x20x1024 maps against a 65536-entry vocabulary: the largest
        {"name": "loss_train_6400_1024_65536", "op": "loss_train", "rows": 6400, "c": 1024, "classes": 65536,
         "ignored": 0.1, "weighted": False},
        # the update of a 3x3x64 -> 64 layer: launches and latency
        {"name": "ortho_64_576", "op": "ortho", "batch": 1, "m": 64, "n": 576, "dtype": "bf16"},
        # six odd, tall matrices at once (heads of 250 channels)
        {"name": "ortho_6x1000_250", "op": "ortho", "batch": 6, "m": 1000, "n": 250, "dtype": "f32"},
        # the update of the 3x3x512 -> 1024 layer: matrix products
        {"name": "ortho_1024_4608", "op": "ortho", "batch": 1, "m": 1024, "n": 4608, "dtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "loss", "loss_train", "ortho"])
    if op in ("norm", "norm_train"):
        cg = rng.choice([1, 2, 4, 5, 8, 10, 12, 16, 20, 32, 64])
        groups = rng.choice([1, 2, 3, 6, 8, 9, 16, 32])
        c = cg * groups
        n = rng.randint(1, 16)
        # at most the largest listed map's values
        most = 16 * 160 * 160 * 128 // (n * c)
        side = _log_int(rng, 1, max(1, min(200, math.isqrt(most))))
        h = side
        w = max(1, min(most // h, side + rng.randint(-3, 3)))
        if h * w * cg < 8:  # a group of a value or two has no spread worth a gradient
            h = w = 3
        dtype = rng.choice(["bf16", "f32"])
        act = rng.choice(["none", "silu", "mish"] + (["relu", "relu6"] if op == "norm" else []))
        return {"op": op, "n": n, "h": h, "w": w, "c": c, "groups": groups,
                "pitch": c + rng.choice([0, 0, 0, 4, 8, c]), "act": act, "dtype": dtype}
    if op in ("loss", "loss_train"):
        rows = _log_int(rng, 1, 6400)
        c = rng.choice([rng.randint(16, 1024), 8 * rng.randint(4, 128), 64 * rng.randint(1, 16)])
        classes = _log_int(rng, 100, 65536)
        return {"op": op, "rows": rows, "c": c, "classes": classes, "ignored": rng.choice([0.0, 0.0, 0.1, 0.5]),
                "weighted": rng.random() < 0.5}
    m, n = _log_int(rng, 8, 2048), _log_int(rng, 8, 4608)
    batch = rng.randint(1, max(1, min(6, 2048 * 4608 // (m * n))))
    return {"op": op, "batch": batch, "m": m, "n": n, "dtype": rng.choice(["bf16", "f32"])}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    op, s = case["op"], dict(case)
    if op in ("norm", "norm_train"):
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        n, h, w, c, pitch = (case[k] for k in ("n", "h", "w", "c", "pitch"))
        # a convolution's output: every channel with an offset and a scale of its own
        x = (randn(n, h, w, pitch) * (0.5 + randn(pitch).abs()) + 0.5 * randn(pitch)).to(dt)
        s["x"] = x[..., :c]
        s["gamma"] = 1.0 + 0.2 * randn(c)
        s["beta"] = 0.2 * randn(c)
        if op == "norm_train":
            s["dy"] = (1e-2 * randn(n, h, w, c)).to(dt)
    elif op in ("loss", "loss_train"):
        rows, c, v = case["rows"], case["c"], case["classes"]
        w = randn(v, c) * (2.0 / math.sqrt(c))
        labels = torch.randint(0, v, (rows,), generator=g, device="cuda")
        # a head in training: the label's logit is raised by about 4 over a spread of 2
        x = randn(rows, c) + w[labels]
        if case["ignored"]:
            out = torch.rand(rows, generator=g, device="cuda") < case["ignored"]
            labels = torch.where(out, torch.full_like(labels, -100), labels)
        s["x"], s["w_head"], s["labels"] = x.bfloat16(), w.bfloat16(), labels
        s["weights"] = (torch.rand(rows, generator=g, device="cuda") + 0.5) / rows if case["weighted"] else None
    else:
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        b, m, n = case["batch"], case["m"], case["n"]
        # a gradient: a few strong directions over a floor of noise
        r = max(1, min(m, n) // 8)
        s["g"] = (1e-3 * (randn(b, m, n) + torch.matmul(randn(b, m, r), randn(b, r, n)) * (2.0 / math.sqrt(r)))).to(dt)
    return s


# ---------------------------------------------------------------- plain forms --

def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "relu6":
        return z.clamp(0.0, 6.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "mish":
        t = torch.exp(z.clamp_max(20.0))
        u = t * (t + 2.0)
        return z * (u / (u + 2.0))
    return z


def _act_slope(z, act):
    if act == "silu":
        q = 1.0 / (1.0 + torch.exp(-z))
        return q * (1.0 + z * (1.0 - q))
    if act == "mish":
        t = torch.exp(z.clamp_max(20.0))
        u = t * (t + 2.0)
        th = u / (u + 2.0)
        return th + z * (1.0 - th * th) * (t / (1.0 + t))
    if act == "relu":
        return (z > 0.0).to(z.dtype)
    if act == "relu6":
        return ((z > 0.0) & (z < 6.0)).to(z.dtype)
    return torch.ones_like(z)


def _norm_plain(s):
    n, h, w, c = s["x"].shape
    k = s["groups"]
    x = s["x"].float().reshape(n, h * w, k, c // k)
    mean = x.mean(dim=(1, 3), keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(dim=(1, 3), keepdim=True) + 1e-5)
    gamma, beta = s["gamma"].view(1, 1, k, c // k), s["beta"].view(1, 1, k, c // k)
    xhat = d * rstd
    z = xhat * gamma + beta
    y = _act(z, s["act"]).reshape(n, h, w, c).to(s["x"].dtype)
    if s["op"] == "norm":
        return y
    dz = s["dy"].float().reshape(n, h * w, k, c // k) * _act_slope(z, s["act"])
    dgamma = (dz * xhat).sum(dim=(0, 1)).reshape(c)
    dbeta = dz.sum(dim=(0, 1)).reshape(c)
    t = dz * gamma
    dx = rstd * (t - t.mean(dim=(1, 3), keepdim=True) - xhat * (t * xhat).mean(dim=(1, 3), keepdim=True))
    return y, dx.reshape(n, h, w, c).to(s["x"].dtype), dgamma, dbeta


def _loss_plain(s):
    labels, v = s["labels"], s["w_head"].shape[0]
    kept = (labels >= 0) & (labels < v)
    at = torch.where(kept, labels, torch.zeros_like(labels))[:, None]
    x, w = torch.where(kept[:, None], s["x"].float(), 0.0), s["w_head"].float()
    weights = s["weights"]
    if weights is None:
        weights = 1.0 / kept.sum().clamp_min(1).float()
    weights = torch.where(kept, weights, 0.0)
    logits = torch.matmul(x, w.t())
    top = logits.amax(dim=1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(dim=1, keepdim=True)
    loss = torch.where(kept, (torch.log(total) - (logits.gather(1, at) - top))[:, 0], 0.0)
    whole = (loss * weights).sum()
    if s["op"] == "loss":
        return whole, loss
    ds = e / total * weights[:, None]
    ds = ds.scatter_add(1, at, -weights[:, None])
    return whole, loss, torch.matmul(ds, w).bfloat16(), torch.matmul(ds.t(), x).bfloat16()


def _ortho_plain(s):
    a, b, c = NS_COEFFS
    x = s["g"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (torch.sqrt((x * x).sum(dim=(1, 2), keepdim=True)) + 1e-7)
    for _ in range(NS_STEPS):
        gram = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return (x.transpose(1, 2) if tall else x).bfloat16().contiguous()


# ------------------------------------------------------------------------ run --

def run(s):
    if not own:
        if s["op"] in ("norm", "norm_train"):
            return _norm_plain(s)
        if s["op"] in ("loss", "loss_train"):
            return _loss_plain(s)
        return _ortho_plain(s)
    import convolution_conv2d_nhwc_amd as conv
    if s["op"] == "norm":
        return conv.group_norm(s["x"], s["groups"], s["gamma"], s["beta"], act=s["act"])
    if s["op"] == "norm_train":
        stats = torch.empty((s["n"], s["groups"], 2), dtype=torch.float32, device="cuda")
        y = conv.group_norm(s["x"], s["groups"], s["gamma"], s["beta"], act=s["act"], stats=stats)
        dx, dgamma, dbeta = conv.group_norm_grad(s["dy"], s["x"], stats, s["gamma"], s["beta"], act=s["act"])
        return y, dx, dgamma, dbeta
    if s["op"] == "loss":
        return conv.head_loss(s["x"], s["w_head"], s["labels"], s["weights"])
    if s["op"] == "loss_train":
        return conv.head_loss_grad(s["x"], s["w_head"], s["labels"], s["weights"])
    return conv.orthogonalize(s["g"], steps=NS_STEPS, coeffs=NS_COEFFS)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_train"):
        e = 2 if case["dtype"] == "bf16" else 4
        values = case["n"] * case["h"] * case["w"] * case["c"]
        if op == "norm":
            return {"bytes": 2 * values * e + 8 * case["c"], "flops": 8 * values}
        return {"bytes": 4 * values * e + 16 * case["c"], "flops": 24 * values}
    if op in ("loss", "loss_train"):
        r, c, v = case["rows"], case["c"], case["classes"]
        if op == "loss":
            return {"bytes": 2 * (r + v) * c + 12 * r, "flops": 2 * r * c * v}
        return {"bytes": 4 * (r + v) * c + 12 * r, "flops": 6 * r * c * v}
    k, n = sorted((case["m"], case["n"]))
    e = 2 if case["dtype"] == "bf16" else 4
    # the two symmetric products of a step need one half of their values
    return {"bytes": case["batch"] * k * n * (e + 2),
            "flops": case["batch"] * NS_STEPS * (k * k * n + k * k * k + 2 * k * k * n)}


# ---------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(s)
    if case["op"] in ("loss", "loss_train"):
        return _exact_loss(s)
    return _exact_ortho(s)


def _exact_norm(s):
    n, h, w, c = s["x"].shape
    k = s["groups"]
    cg = c // k
    # groups to the front: [n, groups, pixels, channels of the group]
    x = s["x"].double().reshape(n, h * w, k, cg).permute(0, 2, 1, 3)
    gamma, beta = (s[p].double().view(1, k, 1, cg) for p in ("gamma", "beta"))
    count = h * w * cg
    mean = x.sum((2, 3), keepdim=True) / count
    var = ((x - mean) ** 2).sum((2, 3), keepdim=True) / count
    dev = torch.sqrt(var + 1e-5)
    xhat = (x - mean) / dev
    z = gamma * xhat + beta
    sig = torch.sigmoid(z)
    th = torch.tanh(torch.logaddexp(z, torch.zeros_like(z)))
    if s["act"] == "silu":
        y, slope = z * sig, sig + z * sig * (1 - sig)
    elif s["act"] == "mish":
        y, slope = z * th, th + z * sig * (1 - th * th)
    elif s["act"] == "relu":
        y, slope = torch.relu(z), (z > 0).double()
    elif s["act"] == "relu6":
        y, slope = z.clamp(0, 6), ((z > 0) & (z < 6)).double()
    else:
        y, slope = z, torch.ones_like(z)

    def back(t):
        return t.permute(0, 2, 1, 3).reshape(n, h, w, c)

    if s["op"] == "norm":
        return back(y)
    dz = s["dy"].double().reshape(n, h * w, k, cg).permute(0, 2, 1, 3) * slope
    u = gamma * dz
    dx = (u - u.sum((2, 3), keepdim=True) / count - xhat * (u * xhat).sum((2, 3), keepdim=True) / count) / dev
    return back(y), back(dx), (dz * xhat).sum((0, 2)).reshape(c), dz.sum((0, 2)).reshape(c)


def _exact_loss(s):
    rows, v = s["x"].shape[0], s["w_head"].shape[0]
    inside = ((s["labels"] >= 0) & (s["labels"] < v)).nonzero()[:, 0]
    x, w, labels = s["x"][inside].double(), s["w_head"].double(), s["labels"][inside]
    if s["weights"] is None:
        weights = torch.full((len(inside),), 1.0 / max(1, len(inside)), dtype=torch.float64, device="cuda")
    else:
        weights = s["weights"][inside].double()
    logp = torch.log_softmax(x @ w.t(), dim=1)
    here = torch.arange(len(inside), device="cuda")
    part = -logp[here, labels]
    loss = torch.zeros(rows, dtype=torch.float64, device="cuda")
    loss[inside] = part
    whole = torch.dot(part, weights)
    if s["op"] == "loss":
        return whole, loss
    d = logp.exp_()
    d[here, labels] -= 1.0
    d *= weights[:, None]
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    dx[inside] = d @ w
    return whole, loss, dx, d.t() @ x


def _exact_ortho(s):
    a, b, c = NS_COEFFS
    out = []
    for g in s["g"].double():
        wide = g if g.shape[0] <= g.shape[1] else g.t()
        x = wide / (wide.norm() + 1e-7)
        for _ in range(NS_STEPS):
            p = x @ x.t()
            px = p @ x
            x = a * x + b * px + c * (p @ px)
        out.append(x if g.shape[0] <= g.shape[1] else x.t())
    return torch.stack(out).contiguous()
