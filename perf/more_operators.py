"""Performance cases of the operators around the attention of a transformer layer.

Three operators, each with its gradients:

* ``layer_norm`` -- layer norm of whole token rows, with the gradients of its weight and bias;
* ``rope``       -- rotation of query and key heads by their positions, without a norm, with frequencies
  scaled for contexts longer than those a model was trained on;
* ``gated_ffn``  -- the gated feed-forward block: two projections, an activation, their product, and the
  projection back.

``run`` computes the plain form (elementary torch operations in 32 bits) or, where ``own`` is true, makes
the calls a user's program makes of this package.  ``exact`` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5
_THETA = 10000.0
# scaled rotations: trained on 8192 tokens, used for 16 times as many
_FACTOR, _TRAINED, _LOW, _HIGH = 16.0, 8192, 1.0, 32.0


# ------------------------------------------------------------------------------------------ cases
def _layer_norm(name, tokens, width, dtype, train, affine=True, sliced=False):
    return {"name": name, "op": "layer_norm", "tokens": tokens, "width": width, "dtype": dtype, "train": train,
            "affine": affine, "sliced": sliced}


def _rope(name, tokens, heads, kv_heads, dim, dtype, train, rot, interleaved=False, fused=False, scaling="none",
          axes=1):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dtype": dtype, "train": train, "rot": rot, "interleaved": interleaved, "fused": fused,
            "scaling": scaling, "axes": axes}


def _gated_ffn(name, tokens, width, hidden, dtype, train, act):
    return {"name": name, "op": "gated_ffn", "tokens": tokens, "width": width, "hidden": hidden, "dtype": dtype,
            "train": train, "act": act}


def listed():
    return [
        # one new token of a model with 32 heads of 128: latency of a single launch
        _layer_norm("layer_norm_one_token", 1, 4096, "bf16", False),
        # fp32 training at an odd length and a width off every power of two
        _layer_norm("layer_norm_f32_train", 4099, 1000, "f32", True),
        # one vision-language sample (2304 image tokens, 16K text) in training
        _layer_norm("layer_norm_vlm_train", 18688, 4096, "bf16", True),
        # the 128K context with 16 heads of 128, forward
        _layer_norm("layer_norm_long", 131072, 2048, "bf16", False),
        # one new token far into a long context, grouped heads, scaled frequencies: latency
        _rope("rope_one_token", 1, 32, 8, 128, "bf16", False, 128, fused=True, scaling="by_parts"),
        # fp32 training, part of each head, neighbouring pairs, odd length
        _rope("rope_f32_train", 4099, 16, 16, 64, "f32", True, 32, interleaved=True),
        # the 128K context with grouped KV heads in training, q and k cut out of one projection's output
        _rope("rope_long_train", 131072, 32, 8, 128, "bf16", True, 128, fused=True, scaling="by_parts"),
        # one new token of a small model: latency
        _gated_ffn("gated_ffn_one_token", 1, 2048, 6144, "bf16", False, "silu"),
        # one new token each of 37 requests: the weights' bytes
        _gated_ffn("gated_ffn_decode", 37, 4096, 12288, "bf16", False, "gelu_tanh"),
        # fp32 training of a small model at an odd length (the precision a gradient check is made in)
        _gated_ffn("gated_ffn_f32_train", 517, 512, 1360, "f32", True, "gelu"),
        # the 8K text sample, forward (evaluation of a loss)
        _gated_ffn("gated_ffn_8k", 8192, 4096, 12288, "bf16", False, "silu"),
        # one vision-language sample (2304 image tokens, 16K text) in training
        _gated_ffn("gated_ffn_vlm_train", 18688, 2048, 8192, "bf16", True, "silu"),
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "rope", "gated_ffn"])
    train = rng.random() < 0.5
    if op == "layer_norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        width = _between(rng, 16, 16384)
        if rng.random() < 0.6:       # most models' widths are multiples of 64
            width = max(64, width // 64 * 64)
        # at most the elements of the largest listed pass
        room = 131072 * 2048 // (width * (2 if dtype == "f32" else 1) * (2 if train else 1))
        return _layer_norm("", _between(rng, 1, max(1, min(131072, room))), width, dtype, train,
                           affine=rng.random() < 0.8, sliced=rng.random() < 0.3)
    if op == "rope":
        dim = rng.choice([64, 128])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        room = 131072 * 40 * 128 // ((heads + kv_heads) * dim * (2 if dtype == "f32" else 1))
        return _rope("", _between(rng, 1, min(131072, room)), heads, kv_heads, dim, dtype, train,
                     rng.choice([dim, dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.3,
                     fused=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "base", "by_parts"]),
                     axes=rng.choice([1, 1, 3]))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    act = rng.choice(["silu", "gelu", "gelu_tanh"])
    # widths are multiples of 8 (16 bytes of bf16), tokens any number
    if dtype == "f32":
        width, hidden = 8 * _between(rng, 4, 96), 8 * _between(rng, 8, 256)
        return _gated_ffn("", _between(rng, 1, 1024), width, hidden, dtype, train, act)
    width, hidden = 8 * _between(rng, 8, 512), 8 * _between(rng, 16, 1536)
    if rng.random() < 0.6:
        width, hidden = max(64, width // 64 * 64), max(128, hidden // 128 * 128)
    room = 18688 * 2048 * 8192 * (1 if train else 3) // (width * hidden)
    return _gated_ffn("", _between(rng, 1, max(1, min(32768, room))), width, hidden, dtype, train, act)


# ------------------------------------------------------------------------------------------ inputs
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _sections(case):
    """Rotated pairs per position axis: all of them, or about a quarter for time and the rest for row and column."""
    pairs = case["rot"] // 2
    if case["axes"] == 1:
        return [pairs]
    time = pairs - 2 * (pairs * 3 // 8)
    return [time, pairs * 3 // 8, pairs * 3 // 8]


def _amplitude(case):
    """The factor that goes with frequencies scaled by parts."""
    return 1.0 + 0.1 * math.log(_FACTOR) if case["scaling"] == "by_parts" else 1.0


def _inputs(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    n = case["tokens"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    if case["op"] == "layer_norm":
        w = case["width"]
        # a residual stream: rows of different size and mean, a few channels far larger than the others
        wide = w + 64 if case["sliced"] else w
        x = normal(n, wide)
        x.mul_(1.0 + 2.0 * torch.rand((n, 1), generator=g, device=dev)).add_(0.3 * normal(n, 1))
        x[:, ::max(1, w // 4)].mul_(12.0)
        return {"x": x.to(dt)[:, wide - w:],
                "w": 1 + 0.2 * normal(w) if case["affine"] else None,
                "b": 0.2 * normal(w) if case["affine"] else None, "dy": normal(n, w).to(dt)}
    if case["op"] == "rope":
        heads, kv, d = case["heads"], case["kv_heads"], case["dim"]
        if case["fused"]:    # one projection's output, [tokens][(q heads, k heads, v heads) x d]
            qkv = normal(n, heads + 2 * kv, d).to(dt)
            q, k = qkv[:, :heads], qkv[:, heads:heads + kv]
        else:
            q, k = normal(n, heads, d).to(dt), normal(n, kv, d).to(dt)
        pos = torch.arange(n, device=dev, dtype=torch.int32)
        if n == 1:
            pos = pos + 100000     # a single token far into its context
        if case["axes"] == 3:      # time for all; rows and columns of 48 x 48 patches in the image part
            image = pos < 2304
            pos = torch.stack([torch.where(image, 0, pos), torch.where(image, pos // 48, pos),
                               torch.where(image, pos % 48, pos)]).to(torch.int32).contiguous()
        return {"q": q, "k": k, "pos": pos, "dq": normal(n, heads, d).to(dt), "dk": normal(n, kv, d).to(dt)}
    d, f = case["width"], case["hidden"]
    # normed rows, and weights that keep their size
    return {"x": normal(n, d).to(dt), "wg": (normal(f, d) * d ** -0.5).to(dt), "wu": (normal(f, d) * d ** -0.5).to(dt),
            "wd": (normal(d, f) * f ** -0.5).to(dt), "dy": normal(n, d).to(dt)}


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if case["op"] == "rope":
        if own:
            import vlm_zigzag_head_gb300 as cp
            state["freq"] = cp.rope_frequencies(case["rot"], _THETA, scaling=case["scaling"], factor=_FACTOR,
                                                trained_length=_TRAINED, low=_LOW, high=_HIGH)
        else:
            state["freq"] = _plain_frequencies(case, state["q"].device)
    return state


def run(state):
    return _RUN[own, state["case"]["op"]](state)


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    n = case["tokens"]
    if case["op"] == "layer_norm":
        # x in, y out; training: dy in, dx out
        elems = n * case["width"]
        return {"bytes": elems * size * (4 if case["train"] else 2) + (8 if case["affine"] else 0) * case["width"],
                "flops": elems * (20 if case["train"] else 8)}
    if case["op"] == "rope":
        elems = n * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": elems * size * (4 if case["train"] else 2) + 4 * n * case["axes"],
                "flops": elems * (6 if case["train"] else 3)}
    d, f = case["width"], case["hidden"]
    weights, rows = 3 * d * f * size, n * d * size
    # x, weights in, y out; training: dy in, dx and the weights' gradients out
    return {"bytes": (2 * weights + 4 * rows) if case["train"] else (weights + 2 * rows),
            "flops": n * d * f * (18 if case["train"] else 6)}


# ------------------------------------------------------------------------------------------ this package's calls
def _own_layer_norm(s):
    import vlm_zigzag_head_gb300 as cp
    y, mean, rstd = cp.cp_layer_norm_fwd(s["x"], s["w"], s["b"], eps=_EPS)
    if not s["case"]["train"]:
        return [y]
    dx, dw, db = cp.cp_layer_norm_bwd(s["x"], s["dy"], mean, rstd, s["w"], bias_grad=s["b"] is not None)
    return [y, dx] + ([dw, db] if s["case"]["affine"] else [])


def _own_rope(s):
    import vlm_zigzag_head_gb300 as cp
    case = s["case"]
    how = dict(rot_dim=case["rot"], sections=_sections(case), interleaved=case["interleaved"], inv_freq=s["freq"],
               amplitude=_amplitude(case))
    out = list(cp.cp_rope_fwd(s["q"], s["k"], s["pos"], **how))
    if case["train"]:
        out += cp.cp_rope_bwd(s["dq"], s["dk"], s["pos"], **how)
    return out


def _own_gated_ffn(s):
    import vlm_zigzag_head_gb300 as cp
    case = s["case"]
    weights = s["wg"], s["wu"], s["wd"]
    if not case["train"]:
        return [cp.cp_gated_ffn_fwd(s["x"], *weights, activation=case["act"])]
    y, gate, up = cp.cp_gated_ffn_fwd(s["x"], *weights, activation=case["act"], keep=True)
    return [y, *cp.cp_gated_ffn_bwd(s["x"], *weights, gate, up, s["dy"], activation=case["act"],
                                    grad_dtype=s["wg"].dtype)]


# ------------------------------------------------------------------------------------------ plain forms
def _plain_layer_norm(s):
    case, x = s["case"], s["x"].float()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    r = torch.rsqrt((c * c).mean(-1, keepdim=True) + _EPS)
    n = c * r
    y = n if s["w"] is None else n * s["w"] + s["b"]
    out = [y.to(s["x"].dtype)]
    if not case["train"]:
        return out
    dy = s["dy"].float()
    g = dy if s["w"] is None else dy * s["w"]
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    out.append(dx.to(s["x"].dtype))
    if case["affine"]:
        # sums over all tokens: in 64 bits
        out += [(dy * n).sum(0, dtype=torch.float64).float(), dy.sum(0, dtype=torch.float64).float()]
    return out


def _plain_frequencies(case, device):
    rot = case["rot"]
    p = torch.arange(0, rot, 2, device=device, dtype=torch.float64)
    theta = _THETA * _FACTOR ** (rot / (rot - 2)) if case["scaling"] == "base" else _THETA
    freq = theta ** (-p / rot)
    if case["scaling"] == "linear":
        freq = freq / _FACTOR
    if case["scaling"] == "by_parts":
        # pairs that turn often within the trained length stay, those that turn less than once are stretched
        stay = ((freq * _TRAINED / (2 * math.pi) - _LOW) / (_HIGH - _LOW)).clamp(0, 1)
        freq = freq * (stay + (1 - stay) / _FACTOR)
    return freq


def _turn_pairs(x, cos, sin, rot, interleaved):
    xf = x.float()
    if interleaved:
        a, b = xf[..., 0:rot:2], xf[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = xf[..., :rot // 2], xf[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, xf[..., rot:]], dim=-1).to(x.dtype)


def _plain_rope(s):
    case = s["case"]
    pos = s["pos"].reshape(case["axes"], -1)
    # angles in 64 bits: a 32-bit angle of a far position is off by whole hundredths of a radian
    axis = torch.tensor([a for a, n in enumerate(_sections(case)) for _ in range(n)], device=pos.device)
    angle = pos[axis].t().to(torch.float64) * s["freq"]
    m = _amplitude(case)
    cos, sin = (m * angle.cos()).float()[:, None], (m * angle.sin()).float()[:, None]
    how = case["rot"], case["interleaved"]
    out = [_turn_pairs(s["q"], cos, sin, *how), _turn_pairs(s["k"], cos, sin, *how)]
    if case["train"]:
        out += [_turn_pairs(s["dq"], cos, -sin, *how), _turn_pairs(s["dk"], cos, -sin, *how)]
    return out


def _plain_activation(g, act):
    """The activation and its derivative."""
    if act == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * 0.5 ** 0.5))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5
    k = (2 / math.pi) ** 0.5
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def _plain_gated_ffn(s):
    case = s["case"]
    dt = s["x"].dtype
    x, wg, wu, wd = (s[name].float() for name in ("x", "wg", "wu", "wd"))
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _plain_activation(g, case["act"])
    h = a * u
    out = [(h @ wd.t()).to(dt)]
    if not case["train"]:
        return out
    dy = s["dy"].float()
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    return out + [(dg @ wg + du @ wu).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt), (dy.t() @ h).to(dt)]


_RUN = {(True, "layer_norm"): _own_layer_norm, (True, "rope"): _own_rope, (True, "gated_ffn"): _own_gated_ffn,
        (False, "layer_norm"): _plain_layer_norm, (False, "rope"): _plain_rope,
        (False, "gated_ffn"): _plain_gated_ffn}


# ------------------------------------------------------------------------------------------ 64-bit values
def exact(case, seed):
    x = _inputs(case, seed)
    return {"layer_norm": _exact_layer_norm, "rope": _exact_rope, "gated_ffn": _exact_gated_ffn}[case["op"]](case, x)


def _exact_layer_norm(case, x):
    """The definition, differentiated by torch; tokens go through in slices, so that the 64-bit copies stay small."""
    n, width, train = case["tokens"], case["width"], case["train"]
    dev = x["x"].device
    w = torch.ones(width, dtype=torch.float64, device=dev) if x["w"] is None else x["w"].double()
    b = torch.zeros(width, dtype=torch.float64, device=dev) if x["b"] is None else x["b"].double()
    w, b = w.requires_grad_(train), b.requires_grad_(train)
    y = torch.empty((n, width), dtype=torch.float64, device=dev)
    dx, dw, db = torch.empty_like(y) if train else None, torch.zeros_like(w), torch.zeros_like(b)
    step = max(1, (1 << 26) // width)
    for t in range(0, n, step):
        rows = x["x"][t:t + step].double().requires_grad_(train)
        spread = rows - rows.sum(1, keepdim=True) / width
        part = spread / (spread.square().sum(1, keepdim=True) / width + _EPS).sqrt() * w + b
        y[t:t + step] = part.detach()
        if train:
            gx, gw, gb = torch.autograd.grad(part, (rows, w, b), x["dy"][t:t + step].double())
            dx[t:t + step] = gx
            dw, db = dw + gw, db + gb
    if not train:
        return [y]
    return [y, dx] + ([dw.detach(), db.detach()] if case["affine"] else [])


def _exact_rope(case, x):
    """Pairs as complex numbers times amplitude exp(i angle); the gradient by the conjugate."""
    rot, inter = case["rot"], case["interleaved"]
    freq = []
    for p in range(rot // 2):
        f = math.exp(-2.0 * p / rot * math.log(_THETA))
        if case["scaling"] == "linear":
            f /= _FACTOR
        elif case["scaling"] == "base":
            f = math.exp(-2.0 * p / rot * (math.log(_THETA) + math.log(_FACTOR) * rot / (rot - 2.0)))
        elif case["scaling"] == "by_parts":
            turns = _TRAINED * f / (2.0 * math.pi)
            share = min(1.0, max(0.0, (turns - _LOW) / (_HIGH - _LOW)))
            f = share * f + (1.0 - share) * f / _FACTOR
        freq.append(f)
    pos = x["pos"].reshape(case["axes"], -1).double()
    parts = torch.split(torch.tensor(freq, dtype=torch.float64, device=pos.device), _sections(case))

    def turned(t, sign):
        out = torch.empty(t.shape, dtype=torch.float64, device=t.device)
        for t0 in range(0, case["tokens"], 16384):
            sl = slice(t0, t0 + 16384)
            angle = sign * torch.cat([pos[a, sl, None] * f for a, f in enumerate(parts)], dim=1)
            v = t[sl].double()
            r = v[..., :rot]
            z = torch.complex(r[..., 0::2], r[..., 1::2]) if inter else \
                torch.complex(r[..., :rot // 2], r[..., rot // 2:])
            z = z * torch.polar(torch.full_like(angle, _amplitude(case)), angle)[:, None]
            r = torch.view_as_real(z).flatten(-2) if inter else torch.cat([z.real, z.imag], -1)
            out[sl] = torch.cat([r, v[..., rot:]], -1)
        return out

    out = [turned(x["q"], 1.0), turned(x["k"], 1.0)]
    return out + ([turned(x["dq"], -1.0), turned(x["dk"], -1.0)] if case["train"] else [])


def _exact_gated_ffn(case, x):
    """Differentiated by torch in 64 bits."""
    if work(case)["flops"] > 7e12:
        return None
    train = case["train"]
    v, wg, wu, wd = (x[name].double().requires_grad_(train) for name in ("x", "wg", "wu", "wd"))
    g = torch.mm(v, wg.t())
    if case["act"] == "silu":
        a = g * torch.sigmoid(g)
    elif case["act"] == "gelu":
        a = g * torch.special.ndtr(g)
    else:
        a = g * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3))
    y = torch.mm(a * torch.mm(v, wu.t()), wd.t())
    if not train:
        return [y]
    return [y.detach(), *torch.autograd.grad(y, (v, wg, wu, wd), x["dy"].double())]
