"""Performance cases of the query / key norm with rotation and of attention with modified scores.

Three operators, each with its gradients:

* ``norm_rope`` -- RMS norm of every query and key head, then the position rotation, in one pass;
* ``scored``    -- packed causal attention whose scores are capped by a tanh and / or get a bias linear
  in the distance, with an image prefix that attends to itself causally or in both directions;
* ``rel_bias``  -- the same attention with a learned bias per head and distance bucket, whose gradient
  is an output of the training pass.

``run`` computes the plain form (elementary torch operations in 32 bits) or, where ``own`` is true, makes
the calls a training program makes of this package.  ``exact`` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_THETA = 10000.0
_EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def _norm_rope(name, tokens, heads, kv_heads, dim, dtype, train, rot, axes=1, interleaved=False, fused=False):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dtype": dtype, "train": train, "rot": rot, "axes": axes, "interleaved": interleaved, "fused": fused}


def _attention(name, op, texts, prefix, heads, kv_heads, dim, dtype, train, scale, cap=0.0, slopes=False,
               both_ways=False, buckets=0, max_distance=0):
    return {"name": name, "op": op, "texts": texts, "prefix": prefix, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "train": train, "scale": scale, "cap": cap, "slopes": slopes,
            "both_ways": both_ways, "buckets": buckets, "max_distance": max_distance}


def listed():
    return [
        # one new token of a grouped-head model: latency of a single launch
        _norm_rope("norm_rope_one_token", 1, 32, 8, 128, "bf16", False, 128),
        # fp32 training at an odd length: half of each head rotated, neighbouring pairs
        _norm_rope("norm_rope_f32_train", 4099, 16, 16, 64, "f32", True, 32, interleaved=True),
        # one vision-language sample (2304 image tokens, 16K text): time / row / column positions, training,
        # q and k cut out of one projection's output
        _norm_rope("norm_rope_vlm_train", 18688, 32, 32, 128, "bf16", True, 128, axes=3, fused=True),
        # the 128K context with grouped KV heads, forward
        _norm_rope("norm_rope_long", 131072, 32, 8, 128, "bf16", False, 128, fused=True),
        # a short prompt with capped scores: latency
        _attention("scored_short", "scored", "33", 0, 4, 4, 64, "bf16", False, 0.125, cap=30.0),
        # the 8K text sample with capped scores, forward (evaluation of a loss)
        _attention("scored_cap_8k", "scored", "8192", 0, 16, 16, 128, "bf16", False, 128 ** -0.5, cap=50.0),
        # packed vision-language samples of ragged lengths: distance bias, the image tokens see one another
        _attention("scored_packed_train", "scored", "1537,6143,2890,1024,4411,999", 576, 16, 4, 128, "bf16", True,
                   128 ** -0.5, slopes=True, both_ways=True),
        # a long vision-language sample with capped scores and grouped KV heads, training
        _attention("scored_long_train", "scored", "16384", 2304, 8, 2, 128, "bf16", True, 128 ** -0.5, cap=50.0,
                   both_ways=True),
        # small fp32 samples (the precision a gradient check is made in), cap and distance bias together
        _attention("scored_f32_train", "scored", "256,129", 17, 4, 2, 64, "f32", True, 0.125, cap=20.0, slopes=True,
                   both_ways=True),
        # a short prompt with a bucketed bias: latency
        _attention("rel_bias_short", "rel_bias", "127", 0, 8, 8, 64, "bf16", False, 0.125, buckets=32,
                   max_distance=128),
        # packed text with softmax scale 1 on queries that carry the scaling, training
        _attention("rel_bias_packed_train", "rel_bias", "2048,1531,700", 0, 12, 12, 64, "bf16", True, 1.0,
                   buckets=32, max_distance=128),
        # a long sample with wide buckets, training
        _attention("rel_bias_long_train", "rel_bias", "12288", 0, 8, 8, 128, "bf16", True, 128 ** -0.5, buckets=64,
                   max_distance=512),
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "scored", "rel_bias"])
    dim = rng.choice([64, 128])
    train = rng.random() < 0.5
    if op == "norm_rope":
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4])
        # the largest listed pass touches about 131072 tokens x 40 heads x 128 elements of two bytes
        dtype = rng.choice(["bf16", "bf16", "f32"])
        room = 131072 * 40 * 128 // ((heads + kv_heads) * dim * (2 if dtype == "f32" else 1) * (2 if train else 1))
        tokens = _between(rng, 1, min(131072, room))
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        return _norm_rope("", tokens, heads, kv_heads, dim, dtype, train, rot, axes=rng.choice([1, 1, 3]),
                          interleaved=rng.random() < 0.3, fused=rng.random() < 0.5)
    dtype = "f32" if rng.random() < 0.15 else "bf16"
    heads, kv_heads = rng.choice([(1, 1), (2, 1), (4, 1), (4, 2), (4, 4), (6, 3), (8, 2), (8, 8)])
    samples = rng.randint(1, 6)
    total = _between(rng, 2 * samples, 768) if dtype == "f32" else _between(rng, 2 * samples, 12000)
    cuts = sorted(rng.randint(0, total) for _ in range(samples - 1))
    texts = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    prefix = rng.choice([0, 0, _between(rng, 1, max(2, total // 4))])
    if dtype == "f32":
        prefix = min(prefix, 64)
    elif prefix * samples > 4000:
        prefix = 4000 // samples
    scale = rng.choice([dim ** -0.5, dim ** -0.5, 1.0])
    cap = rng.choice([0.0, 20.0, 50.0])
    both_ways = prefix > 0 and rng.random() < 0.6
    texts = ",".join(str(t) for t in texts)
    if op == "rel_bias":
        buckets = rng.choice([8, 32, 64])
        return _attention("", op, texts, prefix, heads, kv_heads, dim, dtype, train, scale, cap=cap,
                          both_ways=both_ways, buckets=buckets, max_distance=buckets * rng.choice([2, 4, 8]))
    slopes = cap == 0.0 or rng.random() < 0.5
    return _attention("", op, texts, prefix, heads, kv_heads, dim, dtype, train, scale, cap=cap, slopes=slopes,
                      both_ways=both_ways)


# ------------------------------------------------------------------------------------------ inputs
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _bounds(case):
    """First token of every packed sample [prefix, text], and the end."""
    cu = [0]
    for t in case["texts"].split(","):
        cu.append(cu[-1] + case["prefix"] + int(t))
    return cu


def _sections(case):
    """Rotated pairs per position axis: all of them, or about a quarter for time and the rest for row and column."""
    pairs = case["rot"] // 2
    if case["axes"] == 1:
        return [pairs]
    time = pairs - 2 * (pairs * 3 // 8)
    return [time, pairs * 3 // 8, pairs * 3 // 8]


def _buckets(case):
    """The bucket of every distance 0 .. max_distance: exact below half the buckets, then by logarithm."""
    n, far = case["buckets"], case["max_distance"]
    exact_below = n // 2
    out = []
    for dist in range(far + 1):
        b = dist
        if dist >= exact_below:
            ratio = math.log(dist / exact_below) / math.log(far / exact_below)
            b = min(n - 1, exact_below + int(ratio * (n - exact_below) + 1e-9))
        out.append(b)
    return out


def _inputs(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    heads, kv, d = case["heads"], case["kv_heads"], case["dim"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    if case["op"] == "norm_rope":
        n = case["tokens"]
        if case["fused"]:   # one projection's output, [tokens][(q heads, k heads, v heads) x d]
            qkv = (normal(n, heads + 2 * kv, d) * 1.5).to(dt)
            q, k = qkv[:, :heads], qkv[:, heads:heads + kv]
        else:
            q, k = (normal(n, heads, d) * 1.5).to(dt), (normal(n, kv, d) * 1.5).to(dt)
        pos = torch.arange(n, device=dev, dtype=torch.int32)
        if n == 1:
            pos = pos + 100000   # a single token far into its context
        if case["axes"] == 3:    # time for all; rows and columns of 48 x 48 patches in the image part
            image = pos < 2304
            pos = torch.stack([torch.where(image, 0, pos), torch.where(image, pos // 48, pos),
                               torch.where(image, pos % 48, pos)]).to(torch.int32).contiguous()
        return {"q": q, "k": k, "pos": pos, "qw": 1 + 0.2 * normal(d), "kw": 1 + 0.2 * normal(d),
                "dq": normal(n, heads, d).to(dt), "dk": normal(n, kv, d).to(dt)}
    cu = _bounds(case)
    n = cu[-1]
    # logits of about unit spread; twice that where the scores are capped, so that the cap bends them
    gain = (2.0 if case["cap"] else 1.0) * d ** -0.5 / case["scale"]
    q = (normal(n, heads, d) * gain).to(dt)
    k, v, dout = normal(n, kv, d).to(dt), normal(n, kv, d).to(dt), normal(n, heads, d).to(dt)
    x = {"q": q, "k": k, "v": v, "dout": dout, "slopes": None, "bias": None}
    if case["slopes"]:     # a geometric row of slopes, one per head
        x["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], device=dev)
    if case["buckets"]:
        x["bias"] = (0.5 * normal(heads, case["buckets"])).to(dt)
    return x


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if not own:
        if case["op"] != "norm_rope":
            state["cu"] = _bounds(case)
            if case["buckets"]:
                state["bucket_of"] = torch.tensor(_buckets(case), device=state["q"].device)
        return state
    import vlm_zigzag_head_gb300 as cp
    if case["op"] != "norm_rope":
        # what depends on the packing alone: a training program makes it once per batch, for all layers
        state["plan"] = cp.ScorePlan(_bounds(case), case["heads"], prefix_len=case["prefix"],
                                     bidirectional_prefix=case["both_ways"],
                                     rel_buckets=cp.relative_buckets(case["buckets"], case["max_distance"])
                                     if case["buckets"] else None, device=state["q"].device)
    if case["train"]:
        for name in ("q", "k", "v", "qw", "kw", "bias"):
            if state.get(name) is not None:
                state[name] = state[name].requires_grad_(True)
    return state


def run(state):
    case = state["case"]
    if own:
        return _own_norm_rope(state) if case["op"] == "norm_rope" else _own_attention(state)
    return _plain_norm_rope(state) if case["op"] == "norm_rope" else _plain_attention(state)


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    d, heads, kv = case["dim"], case["heads"], case["kv_heads"]
    if case["op"] == "norm_rope":
        elems = case["tokens"] * (heads + kv) * d
        # q, k in and out; training: the outputs' gradients in, the inputs' gradients out
        passes = 4 if case["train"] else 2
        return {"bytes": elems * size * passes + 4 * case["tokens"] * case["axes"] + 8 * d,
                "flops": elems * (20 if case["train"] else 8)}
    cu = _bounds(case)
    pairs = 0
    for a, b in zip(cu, cu[1:]):
        n = b - a
        pairs += n * (n + 1) // 2
        if case["both_ways"]:
            pairs += case["prefix"] * (case["prefix"] - 1) // 2
    n = cu[-1]
    moved = n * (2 * heads + 2 * kv) * d * size + 4 * heads * n      # q, k, v in; out, lse out
    if case["train"]:
        moved += n * (2 * heads + 2 * kv) * d * size                   # dout in; dq, dk, dv out
    return {"bytes": moved, "flops": pairs * heads * d * (14 if case["train"] else 4)}


# ------------------------------------------------------------------------------------------ this package's calls
def _own_norm_rope(s):
    from vlm_zigzag_head_gb300.autograd import qk_norm_rope
    case = s["case"]
    q, k = qk_norm_rope(s["q"], s["k"], s["pos"], s["qw"], s["kw"], eps=_EPS, theta=_THETA, rot_dim=case["rot"],
                        sections=_sections(case), interleaved=case["interleaved"])
    if not case["train"]:
        return [q, k]
    grads = torch.autograd.grad((q, k), (s["q"], s["k"], s["qw"], s["kw"]), (s["dq"], s["dk"]))
    return [q, k, *grads]


def _own_attention(s):
    from vlm_zigzag_head_gb300.autograd import cp_attention_scored
    case = s["case"]
    out, lse = cp_attention_scored(s["q"], s["k"], s["v"], s["plan"], case["scale"], softcap=case["cap"],
                                   slopes=s["slopes"], rel_bias=s["bias"])
    if not case["train"]:
        return [out, lse]
    leaves = [s["q"], s["k"], s["v"]] + ([s["bias"]] if s["bias"] is not None else [])
    return [out, lse, *torch.autograd.grad(out, leaves, s["dout"])]


# ------------------------------------------------------------------------------------------ plain forms
def _pair_halves(x, rot, interleaved):
    """First and second elements of the rotated pairs, and the elements that are not rotated."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _pair_join(a, b, rest, interleaved):
    if interleaved:
        return torch.cat([torch.stack([a, b], dim=-1).flatten(-2), rest], dim=-1)
    return torch.cat([a, b, rest], dim=-1)


def _plain_norm_rope(s):
    case = s["case"]
    rot, inter = case["rot"], case["interleaved"]
    pos = s["pos"].reshape(case["axes"], -1)
    # angles in 64 bits: a 32-bit angle of a far position is off by whole hundredths of a radian
    axis = torch.tensor([a for a, n in enumerate(_sections(case)) for _ in range(n)], device=pos.device)
    freq = _THETA ** (-torch.arange(0, rot, 2, device=pos.device, dtype=torch.float64) / rot)
    angle = pos[axis].t().to(torch.float64) * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    outs, grads, wgrads = [], [], []
    for x, w, dy in ((s["q"], s["qw"], s["dq"]), (s["k"], s["kw"], s["dk"])):
        xf = x.float()
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + _EPS)
        n = xf * r
        a, b, rest = _pair_halves(n * w, rot, inter)
        outs.append(_pair_join(a * cos - b * sin, b * cos + a * sin, rest, inter).to(x.dtype))
        if case["train"]:
            a, b, rest = _pair_halves(dy.float(), rot, inter)
            g = _pair_join(a * cos + b * sin, b * cos - a * sin, rest, inter)
            wgrads.append((g * n).sum((0, 1)))
            g = g * w
            grads.append((r * (g - n * (g * n).mean(-1, keepdim=True))).to(x.dtype))
    return outs + grads + wgrads


def _diagonal_sums(ds):
    """Sums of ds [h, n, n] over every diagonal: entry n - 1 + (i - j), shape [h, 2 n - 1]."""
    h, n, _ = ds.shape
    # reversing the columns makes i - j + n - 1 the sum of row and column; a row of 2 n elements read as
    # 2 n - 1 shifts each row one place further right
    x = torch.nn.functional.pad(ds.flip(-1), (0, n)).reshape(h, -1)[:, :n * (2 * n - 1)]
    return x.reshape(h, n, 2 * n - 1).sum(1)


def _plain_attention(s):
    case = s["case"]
    q, k, v, dout = s["q"], s["k"], s["v"], s["dout"]
    heads, kv, d = case["heads"], case["kv_heads"], case["dim"]
    group = heads // kv
    scale, cap, cu = case["scale"], case["cap"], s["cu"]
    n = cu[-1]
    out, lse = torch.empty_like(q), torch.empty((heads, n), dtype=torch.float32, device=q.device)
    train, dbias = case["train"], None
    if train:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        if s["bias"] is not None:
            dbias = torch.zeros_like(s["bias"], dtype=torch.float64)
    for b0, b1 in zip(cu, cu[1:]):
        m = b1 - b0
        if m == 0:
            continue
        at = torch.arange(m, device=q.device)
        dist = at[:, None] - at[None, :]
        hidden = dist < 0
        if case["both_ways"]:
            hidden = hidden & ~((at[:, None] < case["prefix"]) & (at[None, :] < case["prefix"]))
        if s["bias"] is not None:
            bucket = s["bucket_of"][dist.abs().clamp(max=case["max_distance"])]
        # as many KV heads at a time as keep one [heads, m, m] matrix near 4 GB
        step = max(1, min(kv, (1 << 30) // max(1, group * m * m)))
        for h0 in range(0, kv, step):
            h1 = min(kv, h0 + step)
            hs = slice(h0 * group, h1 * group)
            qh = q[b0:b1, hs].float().transpose(0, 1)
            kh = k[b0:b1, h0:h1].float().transpose(0, 1).repeat_interleave(group, 0)
            vh = v[b0:b1, h0:h1].float().transpose(0, 1).repeat_interleave(group, 0)
            x = torch.bmm(qh, kh.transpose(1, 2)) * scale
            if cap:
                t = torch.tanh(x / cap)
                x = cap * t
            if s["slopes"] is not None:
                x = x - s["slopes"][hs, None, None] * dist.abs()
            if s["bias"] is not None:
                x = x + s["bias"][hs].float()[:, bucket]
            x = x.masked_fill(hidden, -math.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            total = p.sum(-1, keepdim=True)
            o = torch.bmm(p, vh) / total
            out[b0:b1, hs] = o.transpose(0, 1).to(q.dtype)
            lse[hs, b0:b1] = (top + total.log())[..., 0]
            if not train:
                continue
            p = p / total
            do = dout[b0:b1, hs].float().transpose(0, 1)
            dvh = torch.bmm(p.transpose(1, 2), do)
            ds = p * (torch.bmm(do, vh.transpose(1, 2)) - (do * o).sum(-1, keepdim=True))
            if dbias is not None:
                diag = _diagonal_sums(ds).double()      # [h, 2 m - 1], entry m - 1 is distance 0
                where = s["bucket_of"][(torch.arange(2 * m - 1, device=q.device) - (m - 1)).abs()
                                       .clamp(max=case["max_distance"])]
                dbias[hs] += diag @ (where[:, None] == torch.arange(case["buckets"], device=q.device)).double()
            if cap:
                ds = ds * (1 - t * t)
            ds = ds * scale
            dq[b0:b1, hs] = torch.bmm(ds, kh).transpose(0, 1).to(q.dtype)
            dkh = torch.bmm(ds.transpose(1, 2), qh)
            dk[b0:b1, h0:h1] = dkh.reshape(h1 - h0, group, m, d).sum(1).transpose(0, 1).to(k.dtype)
            dv[b0:b1, h0:h1] = dvh.reshape(h1 - h0, group, m, d).sum(1).transpose(0, 1).to(v.dtype)
    if not train:
        return [out, lse]
    return [out, lse, dq, dk, dv] + ([dbias.to(q.dtype)] if dbias is not None else [])


# ------------------------------------------------------------------------------------------ 64-bit values
def exact(case, seed):
    x = _inputs(case, seed)
    return _exact_norm_rope(case, x) if case["op"] == "norm_rope" else _exact_attention(case, x)


def _exact_norm_rope(case, x):
    """Pairs as complex numbers turned by exp(i angle); gradients by differentiating that.  Tokens go through in
    slices, so that the 64-bit copies stay small."""
    if case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"] > 1 << 30:
        return None
    rot, inter = case["rot"], case["interleaved"]
    pos = x["pos"].reshape(case["axes"], -1).double()
    freq = torch.tensor([_THETA ** (-2.0 * e / rot) for e in range(rot // 2)], dtype=torch.float64, device=pos.device)
    parts = torch.split(freq, _sections(case))
    outs, grads, wgrads = [], [], []
    for name, wname, gname in (("q", "qw", "dq"), ("k", "kw", "dk")):
        y_all = torch.empty(x[name].shape, dtype=torch.float64, device=pos.device)
        dx_all = torch.empty_like(y_all) if case["train"] else None
        w = x[wname].double().requires_grad_(case["train"])
        dw = torch.zeros_like(w)
        for t0 in range(0, case["tokens"], 16384):
            sl = slice(t0, t0 + 16384)
            angle = torch.cat([pos[a, sl, None] * f for a, f in enumerate(parts)], dim=1)
            turn = torch.polar(torch.ones_like(angle), angle)[:, None]
            v = x[name][sl].double().detach().requires_grad_(case["train"])
            n = w * v / (v.square().sum(-1, keepdim=True) / case["dim"] + _EPS).sqrt()
            r = n[..., :rot]
            z = torch.complex(r[..., 0::2], r[..., 1::2]) if inter else torch.complex(r[..., :rot // 2], r[..., rot // 2:])
            z = z * turn
            r = torch.view_as_real(z).flatten(-2) if inter else torch.cat([z.real, z.imag], -1)
            y = torch.cat([r, n[..., rot:]], -1)
            y_all[sl] = y.detach()
            if case["train"]:
                dv, dwi = torch.autograd.grad(y, (v, w), x[gname][sl].double())
                dx_all[sl] = dv
                dw = dw + dwi
        outs.append(y_all)
        if case["train"]:
            grads.append(dx_all)
            wgrads.append(dw.detach())
    return outs + grads + wgrads


def _exact_attention(case, x):
    """One head of one sample at a time, differentiated by torch in 64 bits."""
    if work(case)["flops"] > 8e12:
        return None
    cu = _bounds(case)
    heads, group, train = case["heads"], case["heads"] // case["kv_heads"], case["train"]
    out = torch.zeros(x["q"].shape, dtype=torch.float64, device=x["q"].device)
    lse = torch.zeros((heads, cu[-1]), dtype=torch.float64, device=out.device)
    grads = [torch.zeros(x[n].shape, dtype=torch.float64, device=out.device) for n in "qkv"]
    dbias = torch.zeros(x["bias"].shape, dtype=torch.float64, device=out.device) if x["bias"] is not None else None
    for b0, b1 in zip(cu, cu[1:]):
        m = b1 - b0
        if m == 0:
            continue
        row = torch.arange(m, device=out.device).unsqueeze(1)
        col = row.t()
        seen = col <= row
        if case["both_ways"]:
            seen = seen | (torch.maximum(row, col) < case["prefix"])
        far = (row - col).abs()
        # distance of every pair as an index into the bias by distance
        near = far.clamp(max=case["max_distance"]) if dbias is not None else None
        for h in range(heads):
            q, k, v = (x[n][b0:b1, h if n == "q" else h // group].double().requires_grad_(train) for n in "qkv")
            score = case["scale"] * (q @ k.t())
            if case["cap"]:
                score = case["cap"] * (score / case["cap"]).tanh()
            if x["slopes"] is not None:
                score = score - x["slopes"][h].double() * far
            by_distance = None
            if dbias is not None:
                by_distance = x["bias"][h].double()[torch.tensor(_buckets(case), device=out.device)]
                score = score + by_distance[near]
            score = torch.where(seen, score, -math.inf)
            norm = torch.logsumexp(score, 1)
            prob = torch.exp(score - norm[:, None])
            o = prob @ v
            out[b0:b1, h], lse[h, b0:b1] = o.detach(), norm.detach()
            if not train:
                continue
            wanted = [q, k, v] + ([score] if dbias is not None else [])
            got = torch.autograd.grad(o, wanted, x["dout"][b0:b1, h].double())
            for acc, g, hh in zip(grads, got, (h, h // group, h // group)):
                acc[b0:b1, hh] += g
            if dbias is not None:
                # the gradient of a score is the gradient of its bias: summed over the pairs of a distance
                ds = torch.where(seen, got[3], 0.0)
                for t, b in enumerate(_buckets(case)):
                    if t >= m:
                        break
                    if t < case["max_distance"]:
                        dbias[h, b] += ds.diagonal(-t).sum()
                        if t > 0 and case["both_ways"]:
                            dbias[h, b] += ds.diagonal(t).sum()
                    else:
                        dbias[h, b] += ds.tril(-t).sum() + ds.triu(t).sum()
            del score, prob, got
    if not train:
        return [out, lse]
    return [out, lse, *grads] + ([dbias] if dbias is not None else [])
