"""What is measured of group norm and window attention, the operators that mix voxels' rows.

Beside the convolution, networks on active voxels let rows see each other in
two ways: a norm over all voxels of a frame, and attention inside windows of
voxels with a learned bias for their relative position.

Two operators, each with a serving and a training form:

- group: x_hat = (x - mean) / sqrt(var + eps), y = act(x_hat w + b), mean and variance
  over the rows of a sample and the channels of a group; rows of a batch lie one
  sample after the other (`offsets`). Training returns the statistics too.
- attention: rows are listed window by window (`order`, or as they lie), and
  o_i = sum_j softmax_j(scale q_i k_j + bias_ij) v_j over the window of row i, where
  bias_ij is the sum over the axes of table[axis][clamp(c_i - c_j, -reach, reach)]. Keys
  and values may be shared by groups of heads. Training returns each row's
  log-sum-exp, which the backward pass takes.

`run` takes them through elementary torch operations in float32 where `own` is
false (windows padded to the longest), and through the package's entry points
where it is true.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTIVATIONS = ("none", "relu", "silu", "gelu")


def _group(name, form, dtype, n, c, groups, samples, act):
    return dict(name=name, op="group", form=form, dtype=dtype, n=n, c=c, groups=groups, samples=samples, act=act)


def _attention(name, form, dtype, n, heads, kv_heads, dim, kind, longest, extent=(0, 0, 0), reach=0, order=False):
    return dict(name=name, op="attention", form=form, dtype=dtype, n=n, heads=heads, kv_heads=kv_heads, dim=dim,
                kind=kind, longest=longest, ex=extent[0], ey=extent[1], ez=extent[2], reach=reach, order=order)


def listed():
    return [
        # a frame that has one voxel left at the coarsest stage: latency
        _group("group_single", "serve", "bf16", 1, 512, 32, 1, "silu"),
        # the 91k-voxel stage: a batch of six frames
        _group("group_stage", "serve", "bf16", 91000, 128, 16, 6, "silu"),
        # half precision, odd rows and groups, frames of any size, one without voxels
        _group("group_ragged", "train", "f16", 32371, 200, 10, 9, "gelu"),
        # training on the largest scene: two frames, narrow groups
        _group("group_backward_wide", "backward", "bf16", 95000, 128, 32, 2, "relu"),
        # training the deep stage on a batch of eight
        _group("group_backward_deep", "backward", "bf16", 15000, 512, 32, 8, "silu"),
        # one small window (3 x 3 x 3 cells): latency
        _attention("attention_single", "serve", "bf16", 27, 8, 8, 64, "even", 27, (3, 3, 3), 2),
        # spatial windows of 12 x 12 x 8 cells on the 91k-voxel stage, rows in the convolution's order
        _attention("attention_stage", "serve", "bf16", 91000, 4, 4, 32, "ragged", 160, (12, 12, 8), 11, True),
        # windows of one voxel to a thousand, half precision, head size 24, keys and values shared by three heads
        _attention("attention_ragged", "train", "f16", 32371, 6, 2, 24, "ragged", 1000),
        # every voxel of a frame sees every other: the deep stage, four frames
        _attention("attention_deep", "train", "bf16", 15000, 8, 8, 64, "even", 3750),
        # training a small half-precision scene, wide heads, one set of keys and values
        _attention("attention_backward_small", "backward", "f16", 777, 2, 1, 128, "ragged", 90, (6, 6, 6), 3, True),
        # training the spatial windows of the 91k-voxel stage
        _attention("attention_backward_stage", "backward", "bf16", 91000, 4, 4, 32, "ragged", 160, (12, 12, 8), 11, True),
        # training the deep stage in patches of a serialised order, far distances in one bucket
        _attention("attention_backward_deep", "backward", "bf16", 15000, 8, 8, 64, "even", 1024, (24, 24, 11), 15, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    costs = [work(c) for c in listed()]
    flops, nbytes = max(w["flops"] for w in costs), max(w["bytes"] for w in costs)
    while True:
        form, dtype = rng.choice(("serve", "train", "backward", "backward")), rng.choice(("bf16", "bf16", "f16"))
        if rng.random() < 0.4:
            groups = rng.choice((1, 2, 4, 8, 10, 16, 25, 32))
            case = dict(op="group", form=form, dtype=dtype, n=_log_int(rng, 1, 95000),
                        c=groups * _log_int(rng, 1, max(1, 512 // groups)), groups=groups, samples=_log_int(rng, 1, 16),
                        act=rng.choice(ACTIVATIONS))
            if case["c"] < 8:
                continue
        else:
            kv = rng.choice((1, 2, 4, 8))
            heads = kv * rng.choice((1, 1, 1, 2, 3))
            extent, reach = (0, 0, 0), 0
            if rng.random() < 0.6:
                extent = tuple(_log_int(rng, 2, 40) for _ in range(3))
                reach = _log_int(rng, 1, max(extent))
            case = dict(op="attention", form=form, dtype=dtype, n=_log_int(rng, 1, 95000), heads=heads, kv_heads=kv,
                        dim=rng.choice((16, 24, 32, 32, 48, 64, 64, 96, 128, _log_int(rng, 8, 128))),
                        kind=rng.choice(("even", "ragged")), longest=_log_int(rng, 24, 4000), ex=extent[0],
                        ey=extent[1], ez=extent[2], reach=reach, order=rng.random() < 0.6)
            lengths = _lengths(case)
            # a window holds no cell twice; the plain form's padded scores fit the card
            if sum(extent) and (max(lengths) > math.prod(extent) or sum(extent) > 128):
                continue
            if heads * case["dim"] > 512 or len(lengths) > 8000 or heads * len(lengths) * max(lengths) ** 2 > 1.5e9:
                continue
        w = work(case)
        if w["flops"] <= flops and w["bytes"] <= nbytes:
            return case


def _lengths(case):
    """Rows of each window, or of each sample: the same for every seed, but for their order."""
    n = case["n"]
    if case["op"] == "group":                   # shares of 1, 2, 3, ...; from eight on one sample is empty
        b = case["samples"]
        share = [k + 1 for k in range(b)] if b < 8 else [k for k in range(b)]
        ends = [n * sum(share[:k + 1]) // sum(share) for k in range(b)]
        return [e - (ends[k - 1] if k else 0) for k, e in enumerate(ends)]
    longest, lengths, left, k = case["longest"], [], n, 0
    while left > 0:
        k += 1
        # even: full ones; ragged: spread evenly over the logarithm of 1 .. longest
        length = longest if case["kind"] == "even" else round(longest ** (k * 0.6180339887498949 % 1.0))
        lengths.append(min(left, max(1, length)))
        left -= lengths[-1]
    return lengths


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, n = DTYPES[case["dtype"]], case["n"]

    def normal(shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    lengths = torch.tensor(_lengths(case), device="cuda")
    lengths = lengths[torch.randperm(len(lengths), generator=g, device="cuda")]
    offsets = torch.zeros(len(lengths) + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = lengths.cumsum(0)
    state = dict(case=case, offsets=offsets)
    if case["op"] == "group":
        c = case["c"]
        # a convolution's output: every channel with a mean and a spread of its own
        state["x"] = (normal((n, c)) * (0.5 + torch.rand(c, generator=g, device="cuda")) + normal(c, 0.7)).to(dt)
        state["weight"], state["bias"] = (1 + normal(c, 0.2)).to(dt), normal(c, 0.2).to(dt)
        if case["form"] == "backward":
            state["dy"] = normal((n, c), 0.1).to(dt)
            state["stats"] = _plain_stats(state)
        return state
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    # q, k and v are columns of one projection's output
    qkv = normal((n, (heads + 2 * kv) * dim)).to(dt)
    state["q"], state["k"], state["v"] = qkv.split((heads * dim, kv * dim, kv * dim), 1)
    state["order"] = torch.randperm(n, generator=g, device="cuda").int() if case["order"] else None
    if case["reach"]:
        span = torch.tensor((case["ex"], case["ey"], case["ez"]), device="cuda")
        window = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), lengths)
        corner = torch.randint(0, 1000, (len(lengths), 3), generator=g, device="cuda")[window]
        at = (torch.rand((n, 3), generator=g, device="cuda") * span).long() + corner
        coords = torch.zeros((n, 4), dtype=torch.int32, device="cuda")
        coords[state["order"].long() if case["order"] else slice(None), 1:] = at.int()
        state["coords"] = coords
        state["table"] = normal((3, 2 * case["reach"] + 1, heads), 0.5).to(dt)
    # the window index, made once and kept for every layer of a stage: padded places for the plain form
    first = offsets[:-1].long()
    place = first[:, None] + torch.arange(int(lengths.max()), device="cuda")
    state["inside"] = place < offsets[1:, None]
    place = place.clamp(max=n - 1)
    state["rows"] = state["order"].long()[place] if case["order"] else place
    state["place_of"] = torch.empty(n, dtype=torch.long, device="cuda")     # of each row, in the padded places
    state["place_of"][state["rows"][state["inside"]]] = state["inside"].flatten().nonzero().squeeze(1)
    if own:
        import submanifold_sparse_convolution_amd as smc
        bias = dict(coords=state["coords"], extent=(case["ex"], case["ey"], case["ez"])) if case["reach"] else {}
        state["windows"] = smc.Windows(offsets, n, order=state["order"], **bias)
    if case["form"] == "backward":
        state["dout"] = normal((n, heads * dim), 0.1).to(dt)
        state["out"], state["lse"] = _plain_attention(state, dt)
    return state


# ---- the plain forms ----------------------------------------------------------


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    return torch.ones_like(z)


def _membership(st):
    """[samples, n] float32: 1 where a row is of a sample."""
    at = torch.arange(st["case"]["n"], device="cuda")
    off = st["offsets"]
    return ((at >= off[:-1, None]) & (at < off[1:, None])).float()


def _plain_stats(st):
    x, groups = st["x"].float(), st["case"]["groups"]
    member = _membership(st)
    count = (member.sum(1) * (x.shape[1] // groups)).clamp(min=1)[:, None]
    x = x.view(x.shape[0], groups, -1)
    mean = (member @ x.sum(2)) / count
    off = x - (member.t() @ mean)[:, :, None]
    var = (member @ (off * off).sum(2)) / count
    rstd = torch.where(member.sum(1, keepdim=True) > 0, 1 / torch.sqrt(var + EPS), torch.zeros_like(var))
    return torch.stack((mean, rstd), 2)


def _plain_group(st, dt):
    case = st["case"]
    n, c, groups = case["n"], case["c"], case["groups"]
    stats = st["stats"] if "stats" in st else _plain_stats(st)
    member = _membership(st)
    mean, rstd = (member.t() @ stats[:, :, k] for k in (0, 1))          # of each row
    xhat = ((st["x"].float().view(n, groups, -1) - mean[:, :, None]) * rstd[:, :, None]).view(n, c)
    w = st["weight"].float()
    z = xhat * w + st["bias"].float()
    if case["form"] != "backward":
        y = _act(z, case["act"]).to(dt)
        return (y, stats) if case["form"] == "train" else y
    dz = st["dy"].float() * _act_slope(z, case["act"])
    a = (dz * w).view(n, groups, -1)
    count = (member.sum(1) * (c // groups)).clamp(min=1)[:, None]
    m1 = member.t() @ ((member @ a.sum(2)) / count)
    m2 = member.t() @ ((member @ (a * xhat.view(n, groups, -1)).sum(2)) / count)
    dx = rstd[:, :, None] * (a - m1[:, :, None] - xhat.view(n, groups, -1) * m2[:, :, None])
    return dx.reshape(n, c).to(dt), (dz * xhat).sum(0).to(dt), dz.sum(0).to(dt)


def _padded(t, st, heads):
    """[n, heads dim] -> float32 [windows, heads, longest, dim], zeros where there is no row."""
    t = t.float()[st["rows"]] * st["inside"][:, :, None]
    return t.view(*t.shape[:2], heads, -1).transpose(1, 2)


def _unpadded(t, st, dt):
    """[windows, heads, longest, dim] -> [n, heads dim]."""
    t = t.transpose(1, 2).reshape(-1, t.shape[1] * t.shape[3])
    return t[st["place_of"]].to(dt)


def _cells(st):
    """Each place's cell in its window, [windows, longest, 3]."""
    at = st["coords"][:, 1:].long()[st["rows"]]
    outside = ~st["inside"][:, :, None]
    return (at - at.masked_fill(outside, 1 << 30).amin(1, keepdim=True)).masked_fill(outside, 0)


def _scores(st, q, k):
    case = st["case"]
    s = (q @ k.transpose(2, 3)) * (1 / math.sqrt(case["dim"]))
    if case["reach"]:
        cells, r = _cells(st), case["reach"]
        table = st["table"].float().permute(0, 2, 1)                    # [axis, head, bucket]
        for axis in range(3):
            away = (cells[:, :, None, axis] - cells[:, None, :, axis]).clamp(-r, r) + r
            s = s + table[axis][:, away].transpose(0, 1)
    return s.masked_fill(~st["inside"][:, None, None, :], -math.inf)


def _plain_attention(st, dt):
    case = st["case"]
    heads, kv = case["heads"], case["kv_heads"]
    q, k, v = _padded(st["q"], st, heads), _padded(st["k"], st, kv), _padded(st["v"], st, kv)
    k, v = k.repeat_interleave(heads // kv, 1), v.repeat_interleave(heads // kv, 1)
    s = _scores(st, q, k)
    top = s.amax(3, keepdim=True)
    e = torch.exp(s - top)
    total = e.sum(3, keepdim=True)
    out = _unpadded((e @ v) / total, st, dt)
    lse = (top + torch.log(total)).squeeze(3).transpose(0, 1)           # [heads, windows, longest]
    place = st["place_of"][st["order"].long()] if case["order"] else st["place_of"]
    return out, lse.reshape(heads, -1)[:, place]                        # in the windows' order


def _plain_attention_backward(st, dt):
    case = st["case"]
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    q, k, v = _padded(st["q"], st, heads), _padded(st["k"], st, kv), _padded(st["v"], st, kv)
    k, v = k.repeat_interleave(heads // kv, 1), v.repeat_interleave(heads // kv, 1)
    do = _padded(st["dout"], st, heads)
    s = _scores(st, q, k)
    e = torch.exp(s - s.amax(3, keepdim=True))
    p = e / e.sum(3, keepdim=True) * st["inside"][:, None, :, None]
    dp = do @ v.transpose(2, 3)
    ds = p * (dp - (p * dp).sum(3, keepdim=True))
    scale = 1 / math.sqrt(dim)

    def shared(t):                              # the gradient of a shared head is the sum of its heads'
        return t.view(t.shape[0], kv, heads // kv, t.shape[2], dim).sum(2)

    grads = [_unpadded(ds @ k * scale, st, dt), _unpadded(shared(ds.transpose(2, 3) @ q * scale), st, dt),
             _unpadded(shared(p.transpose(2, 3) @ do), st, dt)]
    if case["reach"]:
        cells, r = _cells(st), case["reach"]
        dtable = torch.zeros((3, 2 * r + 1, heads), device="cuda")
        for axis, extent in enumerate((case["ex"], case["ey"], case["ez"])):
            cell = torch.arange(extent, device="cuda")
            one = ((cells[:, :, axis, None] == cell) & st["inside"][:, :, None]).float()    # [windows, longest, cell]
            by_key = ds @ one[:, None]                                                      # [windows, heads, longest, cell]
            by_both = (one.transpose(1, 2)[:, None] @ by_key).sum(0)                        # [heads, cell, cell of the key]
            away = (cell[:, None] - cell).clamp(-r, r) + r
            bucket = (away.flatten()[None] == torch.arange(2 * r + 1, device="cuda")[:, None]).float()
            dtable[axis] = bucket @ by_both.flatten(1).t()
        grads.append(dtable.to(dt))
    return tuple(grads)


def run(state):
    case = state["case"]
    op, form, dt = case["op"], case["form"], DTYPES[case["dtype"]]
    if not own:
        if op == "group":
            return _plain_group(state, dt)
        if form == "backward":
            return _plain_attention_backward(state, dt)
        out = _plain_attention(state, dt)
        return out if form == "train" else out[0]
    import submanifold_sparse_convolution_amd as smc
    if op == "group":
        x, weight, bias, groups = state["x"], state["weight"], state["bias"], case["groups"]
        if form == "backward":
            return smc.group_norm_backward(state["dy"], x, weight, bias, groups, state["stats"],
                                           offsets=state["offsets"], activation=case["act"])
        return smc.group_norm(x, weight, bias, groups, offsets=state["offsets"], eps=EPS, activation=case["act"],
                              stats=form == "train")
    q, k, v, windows, table = (state.get(t) for t in ("q", "k", "v", "windows", "table"))
    if form == "backward":
        grads = smc.window_attention_backward(state["dout"], q, k, v, state["out"], state["lse"], windows,
                                              case["heads"], bias=table)
        return grads if table is not None else grads[:3]
    return smc.window_attention(q, k, v, windows, case["heads"], bias=table, lse=form == "train")


def work(case):
    """Each input read once, each output written once; 2 operations a product term."""
    n, back = case["n"], case["form"] == "backward"
    if case["op"] == "group":
        c = case["c"]
        stats = 8 * case["groups"] * case["samples"] if case["form"] != "serve" else 0
        return dict(bytes=n * c * (6 if back else 4) + stats + c * (8 if back else 4), flops=n * c * (16 if back else 10))
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    pairs = sum(length * length for length in _lengths(case))
    c, ckv = heads * dim, kv * dim
    moved = 2 * n * (4 * c + 4 * ckv) if back else 2 * n * (2 * c + 2 * ckv)   # backward: out, dout, dq and dk, dv too
    moved += 4 * n * heads if case["form"] != "serve" else 0
    moved += (4 * n if case["order"] else 0) + (12 * n + 6 * (2 * case["reach"] + 1) * heads if case["reach"] else 0)
    return dict(bytes=moved, flops=pairs * c * (10 if back else 4))


# ---- the definition, in 64 bits -----------------------------------------------


def _window_of(case, rows, coords, q, k, v, table):
    """Scores [heads, L, L] and values [heads, L, dim] of one window's rows."""
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    q = q.view(-1, heads, dim).permute(1, 0, 2)
    k, v = (torch.stack([t.view(-1, kv, dim)[:, h * kv // heads] for h in range(heads)]) for t in (k, v))
    s = torch.bmm(q, k.permute(0, 2, 1).contiguous()) / math.sqrt(dim)
    if case["reach"]:
        at = coords[rows, 1:].long()
        apart = torch.clamp(at[:, None] - at[None], min=-case["reach"], max=case["reach"]) + case["reach"]
        bias = table[0][apart[..., 0]] + table[1][apart[..., 1]] + table[2][apart[..., 2]]
        s = s + bias.movedim(2, 0)
    return s, v


def _exact_group(st, off):
    case = st["case"]
    back = case["form"] == "backward"
    x, w, b = (st[t].double().requires_grad_(back) for t in ("x", "weight", "bias"))
    f = {"none": lambda t: t, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": torch.nn.functional.gelu}[case["act"]]
    y, stats = [], torch.zeros((len(off) - 1, case["groups"], 2), dtype=torch.float64, device="cuda")
    for k, (begin, end) in enumerate(zip(off[:-1], off[1:])):
        if begin == end:
            continue
        part = x[begin:end].reshape(end - begin, case["groups"], -1)
        var, mean = torch.var_mean(part, dim=(0, 2), unbiased=False, keepdim=True)
        y.append(((part - mean) * torch.rsqrt(var + EPS)).reshape(end - begin, -1))
        stats[k] = torch.stack((mean, torch.rsqrt(var + EPS)), 3).detach().view(-1, 2)
    y = f(torch.cat(y) * w + b)
    if back:
        return torch.autograd.grad(y, (x, w, b), st["dy"].double())
    return (y, stats) if case["form"] == "train" else y


def exact(case, seed):
    st = prepare(case, seed)
    off = st["offsets"].tolist()
    if case["op"] == "group":
        return _exact_group(st, off)
    back, n = case["form"] == "backward", case["n"]
    q, k, v = (st[t].double() for t in ("q", "k", "v"))
    table = st["table"].double().requires_grad_(back) if case["reach"] else None
    out, lse = torch.zeros_like(q), torch.zeros((case["heads"], n), dtype=torch.float64, device="cuda")
    grads = [torch.zeros_like(t) for t in (q, k, v)] + ([torch.zeros_like(table)] if case["reach"] else [])
    for begin, end in zip(off[:-1], off[1:]):
        rows = st["order"][begin:end].long() if case["order"] else torch.arange(begin, end, device="cuda")
        own_rows = [t[rows].requires_grad_(back) for t in (q, k, v)]
        s, val = _window_of(case, rows, st.get("coords"), *own_rows, table)
        o = torch.bmm(torch.softmax(s, 2), val).permute(1, 0, 2).reshape(end - begin, -1)
        if back:
            got = torch.autograd.grad(o, own_rows + ([table] if case["reach"] else []), st["dout"][rows].double())
            for total, g in zip(grads[:3], got):
                total[rows] = g
            if case["reach"]:
                grads[3] += got[3]
        else:
            out[rows] = o
            lse[:, begin:end] = torch.logsumexp(s, 2)
    if back:
        return tuple(grads)
    return (out, lse) if case["form"] == "train" else out
