"""The transformer-block operators on real shapes: cases, inputs, plain forms and exact values.

Three operators, each with its directions:

  layer_norm   rows of a token matrix normalised over their last axis; forward (Y, Mean,
               InvStdDev) and backward (dX, dScale, dB).
  dropout      residual + dropout(X) with the mask drawn from a counter-based generator
               (Philox4x32-10); the backward pass is the same call on the gradient.
  attention    softmax(scale Q K^T + table[bucket(relative position)]) V over tokens that
               lie on a grid; forward (O, LSE) and backward (dQ, dK, dV, dTable).

With ``own`` false, ``run`` computes the plain form in elementary torch operations and 32 bits,
rounded once at the end; with ``own`` true it makes the calls of the package.
"""
import math

import torch

own = False

DT = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
EPS = 1e-5


# ------------------------------------------------------------------ cases

def _ln(name, direction, dtype, rows, width):
    return {"name": name, "op": "layer_norm", "dir": direction, "dtype": dtype, "rows": rows,
            "width": width}


def _drop(name, direction, dtype, rows, width, ratio):
    return {"name": name, "op": "dropout", "dir": direction, "dtype": dtype, "rows": rows,
            "width": width, "ratio": ratio}


def _attn(name, direction, dtype, N, H, D, q, k, buckets, ragged):
    return {"name": name, "op": "attention", "dir": direction, "dtype": dtype, "N": N, "H": H,
            "D": D, "qh": q[0], "qw": q[1], "kh": k[0], "kw": k[1], "buckets": buckets,
            "ragged": ragged}


def listed():
    return [
        # the pooled token of a few images before a classifier: latency only
        _ln("ln_fwd_few_rows", "forward", "bfloat16", 7, 384),
        # every pixel of a 16 x 64 x 256 x 256 feature map as a token of 64 channels
        _ln("ln_fwd_pixels", "forward", "float32", 16 * 256 * 256, 64),
        # a training step's tokens at a wide model width
        _ln("ln_bwd_wide", "backward", "bfloat16", 16384, 1024),
        # odd rows and width: nothing divides a vector or a tile
        _ln("ln_bwd_odd", "backward", "float32", 5003, 771),
        # branch dropout and residual of one small batch of 24 x 24 grids
        _drop("dropout_small", "forward", "float32", 577, 33, 0.1),
        # the same over a 16 x 64 x 256 x 256 map
        _drop("dropout_large", "forward", "bfloat16", 16 * 256 * 256, 64, 0.1),
        # gradient of the branch
        _drop("dropout_bwd", "backward", "float16", 32768, 1024, 0.25),
        # 8 x 8 windows of a 128 x 128 map for a batch of 4, a bias entry per offset
        _attn("attn_windows", "forward", "bfloat16", 1024, 4, 32, (8, 8), (8, 8), "each", False),
        # global attention over the 64 x 64 map, logarithmic buckets per axis
        _attn("attn_map", "forward", "float16", 8, 8, 64, (64, 64), (64, 64), "log", False),
        # one new token against a long memory of ragged length
        _attn("attn_single", "forward", "bfloat16", 8, 8, 64, (1, 1), (1, 32771), "log", True),
        # training at 32 x 32 tokens, ragged batch
        _attn("attn_train", "backward", "bfloat16", 8, 8, 64, (32, 32), (32, 32), "log", True),
        # training in 32 bits on an odd grid
        _attn("attn_train_odd", "backward", "float32", 4, 4, 48, (17, 23), (17, 23), "each", True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layer_norm", "dropout", "attention", "attention"])
    dtype = rng.choice(list(DT))
    direction = rng.choice(["forward", "backward"])
    if op == "layer_norm":
        width = _logint(rng, 16, 8192)
        rows = _logint(rng, 1, min(16 * 256 * 256, (1 << 25) // width))
        return {"op": op, "dir": direction, "dtype": dtype, "rows": rows, "width": width}
    if op == "dropout":
        width = _logint(rng, 16, 4096)
        rows = _logint(rng, 1, min(16 * 256 * 256, (1 << 25) // width))
        return {"op": op, "dir": direction, "dtype": dtype, "rows": rows, "width": width,
                "ratio": round(rng.uniform(0.0, 0.5), 3)}
    kind = rng.choice(["window", "map", "sequence", "single"])
    H = rng.choice([1, 2, 3, 4, 6, 8, 12])
    D = rng.choice([16, 24, 32, 40, 48, 64, 80, 96, 128])
    if kind == "window":
        q = k = (rng.randint(4, 14), rng.randint(4, 14))
        N = _logint(rng, 16, 1024)
    elif kind == "map":
        q = k = (_logint(rng, 9, 48), _logint(rng, 9, 48))
        N = rng.randint(1, 8)
    elif kind == "sequence":
        length = _logint(rng, 2, 3000)
        q = k = (1, length)
        N = rng.randint(1, 4)
    else:
        q, k = (1, 1), (1, _logint(rng, 1, 32768))
        N = rng.randint(1, 8)
        direction = "forward"
    each = (4 if direction == "forward" else 10) * H * D * (q[0] * q[1]) * (k[0] * k[1])
    N = max(1, min(N, 275_000_000_000 // each))
    return {"op": op, "dir": direction, "dtype": dtype, "N": N, "H": H, "D": D, "qh": q[0],
            "qw": q[1], "kh": k[0], "kw": k[1], "buckets": rng.choice(["each", "log"]),
            "ragged": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _axis_buckets(offsets, num, far):
    """Buckets of signed offsets (query minus key): `num` // 2 per sign, the first half of them
    one offset each, the rest spaced by a constant ratio up to `far`."""
    half = num // 2
    near = half // 2
    ratio = far / near
    first = list(range(1, near + 1)) + [math.ceil(near * ratio ** (k / (half - near)) - 1e-9)
                                        for k in range(1, half - near)]
    offsets = torch.tensor(offsets)
    b = torch.bucketize(offsets.abs(), torch.tensor(first), right=True)
    return b + torch.where(offsets < 0, half, 0)


def _bucket_map(case):
    """int32 map of relative grid positions to rows of the bias table, and the table's rows."""
    qh, qw, kh, kw = (case[x] for x in ("qh", "qw", "kh", "kw"))
    nh, nw = qh + kh - 1, qw + kw - 1
    if case["buckets"] == "each":
        return torch.arange(nh * nw, dtype=torch.int32), nh * nw
    # a lone query stands at the last key
    oy, ox = (kh - 1 if qh == 1 else 0), (kw - 1 if qw == 1 else 0)
    wide, far = (16, 64) if nh > 1 else (32, 1024)
    ys = _axis_buckets([a - (kh - 1) + oy for a in range(nh)], 16, 64)
    xs = _axis_buckets([a - (kw - 1) + ox for a in range(nw)], wide, far)
    m = ys.view(-1, 1) * (wide if nh > 1 else 0) + xs.view(1, -1)
    return m.reshape(-1).to(torch.int32), 16 * wide if nh > 1 else wide


def prepare(case, seed):
    g = _gen(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dt)

    s = {"case": dict(case)}
    if case["op"] == "layer_norm":
        rows, width = case["rows"], case["width"]
        level = torch.randn((rows, 1), generator=g, device="cuda")
        X = (torch.randn((rows, width), generator=g, device="cuda") * 1.5 + level).to(dt)
        s.update(X=X, Scale=normal(width, std=0.2, mean=1.0), B=normal(width, std=0.2))
        if case["dir"] == "backward":
            X32 = X.float()
            mean = X32.mean(1, keepdim=True)
            var = (X32 - mean).square().mean(1, keepdim=True)
            s.update(dY=normal(rows, width), Mean=mean, InvStdDev=1.0 / torch.sqrt(var + EPS))
        return s
    if case["op"] == "dropout":
        shape = (case["rows"], case["width"])
        s.update(X=normal(*shape), seed=(0x9E3779B97F4A7C15 * (seed + 1)) % (1 << 63),
                 offset=seed % 1000)
        if case["dir"] == "forward":
            s["residual"] = normal(*shape)
        return s
    N, H, D = case["N"], case["H"], case["D"]
    Lq, Lk = case["qh"] * case["qw"], case["kh"] * case["kw"]
    if Lq == Lk:                      # one projection's output, heads inside
        qkv = normal(N, Lq, 3, H, D)
        Q, K, V = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    else:                             # a new token and the kept keys and values
        Q, kv = normal(N, Lq, H, D), normal(N, Lk, 2, H, D)
        K, V = kv[:, :, 0], kv[:, :, 1]
    buckets, nb = _bucket_map(case)
    s.update(Q=Q, K=K, V=V, table=normal(nb, H, std=0.7), buckets=buckets.cuda(), k_len=None,
             scale=1.0 / math.sqrt(D), q_extent=(case["qh"], case["qw"]),
             k_extent=(case["kh"], case["kw"]))
    if case["ragged"]:
        k_len = torch.randint(max(1, Lk // 2), Lk + 1, (N,), generator=g, device="cuda")
        s["k_len"] = k_len.to(torch.int32)
    if case["dir"] == "backward":
        s["dO"] = normal(N, Lq, H, D)
        s["O"], s["LSE"] = _attention_plain(s)
    return s


# ------------------------------------------------------------------ plain forms

def _layer_norm_plain(s):
    X, dt = s["X"].float(), s["X"].dtype
    mean = X.mean(1, keepdim=True)
    d = X - mean
    inv = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    return (d * inv * s["Scale"].float() + s["B"].float()).to(dt), mean, inv


def _layer_norm_backward_plain(s):
    dt = s["X"].dtype
    dY, inv = s["dY"].float(), s["InvStdDev"]
    xhat = (s["X"].float() - s["Mean"]) * inv
    g = dY * s["Scale"].float()
    dX = inv * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dX.to(dt), (dY * xhat).sum(0).to(dt), dY.sum(0).to(dt)


def _philox_words(n, seed, offset, device):
    """The first n 32-bit words of the generator, as int64 (Philox4x32-10; the low 64 bits of an
    int64 product are those of the unsigned one)."""
    low = 0xFFFFFFFF
    i = torch.arange((n + 3) // 4, device=device)
    c0, c1 = i & low, i >> 32
    c2, c3 = torch.full_like(i, offset & low), torch.full_like(i, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((p1 >> 32) & low) ^ c1 ^ k0, p1 & low,
                          ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((c0, c1, c2, c3), 1).reshape(-1)[:n]


def _dropout_plain(s):
    X, ratio = s["X"], s["case"]["ratio"]
    words = _philox_words(X.numel(), s["seed"], s["offset"], X.device).view(X.shape)
    keep = words >= int(math.floor(ratio * 4294967296.0 + 0.5))
    Y = torch.where(keep, X.float() * (1.0 / (1.0 - ratio)), 0.0)
    if "residual" in s:
        Y = s["residual"].float() + Y
    return Y.to(X.dtype)


def _relative_index(s):
    (qh, qw), (kh, kw) = s["q_extent"], s["k_extent"]
    i = torch.arange(qh * qw, device="cuda").view(-1, 1)
    j = torch.arange(kh * kw, device="cuda").view(1, -1)
    dy = torch.div(i, qw, rounding_mode="floor") - torch.div(j, kw, rounding_mode="floor") + kh - 1
    return dy * (qw + kw - 1) + i % qw - j % kw + kw - 1


def _scores(s):
    """(N, H, Lq, Lk) scaled and biased scores, -inf where masked, and the bucket of each pair."""
    Q, K = s["Q"].float().permute(0, 2, 1, 3), s["K"].float().permute(0, 2, 3, 1)
    b = s["buckets"].long()[_relative_index(s)]
    S = torch.matmul(Q, K) * s["scale"] + s["table"].float()[b].permute(2, 0, 1)
    if s["k_len"] is not None:
        dead = torch.arange(K.shape[3], device="cuda").view(1, -1) >= s["k_len"].view(-1, 1)
        S = S.masked_fill(dead[:, None, None, :], -math.inf)
    return S, b


def _attention_plain(s):
    S, _ = _scores(s)
    top = S.amax(3, keepdim=True)
    P = torch.exp(S - top)
    total = P.sum(3, keepdim=True)
    O = torch.matmul(P / total, s["V"].float().permute(0, 2, 1, 3))
    LSE = (top + torch.log(total)).squeeze(3)
    return O.permute(0, 2, 1, 3).contiguous().to(s["Q"].dtype), LSE


def _attention_backward_plain(s):
    dt = s["Q"].dtype
    S, b = _scores(s)
    Q, K, V, dO, O = (s[x].float().permute(0, 2, 1, 3) for x in ("Q", "K", "V", "dO", "O"))
    P = torch.exp(S - s["LSE"].unsqueeze(3))
    dP = torch.matmul(dO, V.transpose(2, 3))
    dS = P * (dP - (dO * O).sum(3, keepdim=True))
    back = [torch.matmul(dS, K) * s["scale"], torch.matmul(dS.transpose(2, 3), Q) * s["scale"],
            torch.matmul(P.transpose(2, 3), dO)]
    per_pair = dS.sum(0).permute(1, 2, 0).reshape(-1, Q.shape[1])
    dT = torch.zeros(s["table"].shape, device="cuda").index_add_(0, b.reshape(-1), per_pair)
    return [x.permute(0, 2, 1, 3).contiguous().to(dt) for x in back] + [dT.to(dt)]


# ------------------------------------------------------------------ one pass

def run(s):
    op, forward = s["case"]["op"], s["case"]["dir"] == "forward"
    if not own:
        if op == "layer_norm":
            return _layer_norm_plain(s) if forward else _layer_norm_backward_plain(s)
        if op == "dropout":
            return _dropout_plain(s)
        return _attention_plain(s) if forward else _attention_backward_plain(s)
    import spatial_transformer_sampling_gb300 as gs
    if op == "layer_norm":
        if forward:
            return gs.gs_layer_norm(s["X"], s["Scale"], s["B"], epsilon=EPS)
        return gs.gs_layer_norm_backward(s["dY"], s["X"], s["Scale"], s["Mean"], s["InvStdDev"])
    if op == "dropout":
        return gs.gs_dropout(s["X"], s["case"]["ratio"], s["seed"], s["offset"],
                             residual=s.get("residual"))
    bias = dict(table=s["table"], buckets=s["buckets"], q_extent=s["q_extent"],
                k_extent=s["k_extent"], k_len=s["k_len"], scale=s["scale"])
    if forward:
        return gs.gs_attention(s["Q"], s["K"], s["V"], **bias)
    return gs.gs_attention_backward(s["dO"], s["Q"], s["K"], s["V"], s["O"], s["LSE"], **bias)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    e = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "layer_norm":
        n, rows, width = case["rows"] * case["width"], case["rows"], case["width"]
        if case["dir"] == "forward":
            return {"bytes": 2 * n * e + 2 * width * e + 8 * rows, "flops": 8 * n}
        return {"bytes": 3 * n * e + 3 * width * e + 8 * rows, "flops": 14 * n}
    if case["op"] == "dropout":
        n = case["rows"] * case["width"]
        return {"bytes": (3 if case["dir"] == "forward" else 2) * n * e, "flops": 2 * n}
    N, H, D = case["N"], case["H"], case["D"]
    Lq, Lk = case["qh"] * case["qw"], case["kh"] * case["kw"]
    live = 0.75 if case["ragged"] else 1.0   # lengths are uniform between half and all
    q, k = N * Lq * H * D, N * Lk * H * D * live
    bias = 4 * (case["qh"] + case["kh"] - 1) * (case["qw"] + case["kw"] - 1)
    pairs = N * H * Lq * Lk * live
    if case["dir"] == "forward":
        return {"bytes": (2 * q + 2 * k) * e + bias + 4 * N * H * Lq, "flops": 4 * pairs * D}
    return {"bytes": (4 * q + 4 * k) * e + bias + 4 * N * H * Lq, "flops": 10 * pairs * D}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "layer_norm":
        x = s["X"].to(f64)
        if case["dir"] == "forward":
            mean = x.sum(1, keepdim=True) / x.shape[1]
            inv = (((x - mean) ** 2).sum(1, keepdim=True) / x.shape[1] + EPS).rsqrt()
            return (x - mean) * inv * s["Scale"].to(f64) + s["B"].to(f64), mean, inv
        dy, mean, inv = s["dY"].to(f64), s["Mean"].to(f64), s["InvStdDev"].to(f64)
        xh, w, D = (x - mean) * inv, s["Scale"].to(f64), x.shape[1]
        a = (dy * w).sum(1, keepdim=True)
        b = (dy * w * xh).sum(1, keepdim=True)
        return (dy * w * D - a - xh * b) * inv / D, (dy * xh).sum(0), dy.sum(0)
    if case["op"] == "dropout":
        n = s["X"].numel()
        m16 = 0xFFFF

        def mul(a, m):   # 32 x 32 -> (high, low) words from 16-bit halves
            lo, hi = a * (m & m16), a * (m >> 16)
            mid = hi + (lo >> 16)
            return mid >> 16, ((mid & m16) << 16) | (lo & m16)

        idx = torch.arange((n + 3) // 4, device="cuda")
        ctr = [idx % (1 << 32), idx // (1 << 32), torch.zeros_like(idx) + s["offset"] % (1 << 32),
               torch.zeros_like(idx) + s["offset"] // (1 << 32)]
        for rnd in range(10):
            ka = (s["seed"] % (1 << 32) + rnd * 0x9E3779B9) % (1 << 32)
            kb = (s["seed"] // (1 << 32) + rnd * 0xBB67AE85) % (1 << 32)
            h0, l0 = mul(ctr[0], 0xD2511F53)
            h1, l1 = mul(ctr[2], 0xCD9E8D57)
            ctr = [h1 ^ ctr[1] ^ ka, l1, h0 ^ ctr[3] ^ kb, l0]
        words = torch.stack(ctr, 1).reshape(-1)[:n].view(s["X"].shape)
        kept = (words >= round(case["ratio"] * 2 ** 32)).to(f64)
        y = s["X"].to(f64) * kept / (1.0 - case["ratio"])
        return y + s["residual"].to(f64) if "residual" in s else y
    N, Lq, H, D = s["Q"].shape
    Lk = s["K"].shape[1]
    yq, xq = [t.reshape(-1) for t in torch.meshgrid(torch.arange(case["qh"], device="cuda"),
                                                    torch.arange(case["qw"], device="cuda"),
                                                    indexing="ij")]
    yk, xk = [t.reshape(-1) for t in torch.meshgrid(torch.arange(case["kh"], device="cuda"),
                                                    torch.arange(case["kw"], device="cuda"),
                                                    indexing="ij")]
    grid = s["buckets"].view(case["qh"] + case["kh"] - 1, case["qw"] + case["kw"] - 1)
    which = grid[yq[:, None] - yk[None, :] + case["kh"] - 1,
                 xq[:, None] - xk[None, :] + case["kw"] - 1].long()
    forward = case["dir"] == "forward"
    O = torch.zeros((N, Lq, H, D), dtype=f64, device="cuda")
    LSE = torch.zeros((N, H, Lq), dtype=f64, device="cuda")
    dQ = torch.zeros((N, Lq, H, D), dtype=f64, device="cuda")
    dK, dV = (torch.zeros((N, Lk, H, D), dtype=f64, device="cuda") for _ in range(2))
    dT = torch.zeros(s["table"].shape, dtype=f64, device="cuda")
    for h in range(H):
        bias = s["table"][:, h].to(f64)[which]
        total = torch.zeros((Lq, Lk), dtype=f64, device="cuda")
        for n in range(N):
            m = Lk if s["k_len"] is None else int(s["k_len"][n])
            q, k, v = s["Q"][n, :, h].to(f64), s["K"][n, :m, h].to(f64), s["V"][n, :m, h].to(f64)
            a = q @ k.T * s["scale"] + bias[:, :m]
            if forward:
                LSE[n, h] = torch.logsumexp(a, 1)
                O[n, :, h] = torch.exp(a - LSE[n, h][:, None]) @ v
                continue
            do = s["dO"][n, :, h].to(f64)
            p = torch.exp(a - s["LSE"][n, h].to(f64)[:, None])
            ds = p * (do @ v.T - (do * s["O"][n, :, h].to(f64)).sum(1, keepdim=True))
            dQ[n, :, h], dK[n, :m, h] = ds @ k * s["scale"], ds.T @ q * s["scale"]
            dV[n, :m, h] = p.T @ do
            total[:, :m] += ds
        if not forward:
            dT[:, h].index_add_(0, which.reshape(-1), total.reshape(-1))
    return (O, LSE) if forward else [dQ, dK, dV, dT]
