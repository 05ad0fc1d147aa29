"""Cases that measure the operators between two attention layers' projections.

Four operators of the feed-forward half of a layer: the addition of the
residual with its root-mean-square norm and the 8-bit codes that the next
product reads (``norm``), the choice of experts (``route``), the product of
8-bit activations with a 4-bit weight (``linear``), and the routed experts on
4-bit weights: gate and up product, SwiGLU, down product, weighted sum
(``experts``).  Codes are OCP E4M3 with an E8M0 scale per 128 values; 4-bit
weights are OCP E2M1 with an E8M0 scale per 32.

``own`` selects what ``run`` computes: the plain form (elementary torch
operations in 32 bits, 64 where experts are compared) or the library's entry
points.
"""

import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # The norm in front of one decode step's projection: latency only.
        dict(name="norm 1x4096", op="norm", T=1, D=4096, residual=True, y=False, codes=True),
        # Per-head norms of a batch's queries: many short rows, no residual, BF16 alone.
        dict(name="norm 4160x512 heads", op="norm", T=4160, D=512, residual=False, y=True, codes=False),
        # The 8192-token prefill chunk: the sum, the BF16 form for a router and the codes for the products.
        dict(name="norm 8192x4096", op="norm", T=8192, D=4096, residual=True, y=True, codes=True),
        # One token's experts: sigmoid scores, balance bias, 4 of 8 groups.
        dict(name="route 1x256", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4, bf16=False),
        # A ragged batch over an odd number of experts, softmax, scores straight from a BF16 product.
        dict(name="route 777x60 softmax", op="route", T=777, E=60, k=6, score="softmax", bias=False, groups=1, keep=1,
             bf16=True),
        # The prefill chunk's routing.
        dict(name="route 8192x256", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4,
             bf16=False),
        # One token through a square projection: the weight's bytes are the time.
        dict(name="linear 1x4096x4096", op="linear", T=1, N=4096, K=4096),
        # A decode batch through a down projection whose shard is no multiple of 128 columns.
        dict(name="linear 48x5120x576", op="linear", T=48, N=5120, K=576),
        # A prefill chunk: products are the time.
        dict(name="linear 2048x4096x4096", op="linear", T=2048, N=4096, K=4096),
        # One token's eight experts out of 128.
        dict(name="experts 1 of 128x1024", op="experts", T=1, E=128, k=8, K=4096, I=1024, pad=False),
        # A decode batch with padded rows: nearly every expert is read, for a few rows each.
        dict(name="experts 64 of 128x1024", op="experts", T=64, E=128, k=8, K=4096, I=1024, pad=True),
        # A prefill chunk: hundreds of rows for each expert, unevenly.
        dict(name="experts 4096 of 64x1024", op="experts", T=4096, E=64, k=6, K=4096, I=1024, pad=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "linear", "linear", "experts", "experts"])
    if op == "norm":
        T, D = _log(rng, 1, 8192), 16 * _log(rng, 2, 512)
        y = rng.random() < 0.7
        return dict(op=op, T=min(T, 8192 * 4096 // D), D=D, residual=rng.random() < 0.7, y=y,
                    codes=not y or rng.random() < 0.5)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 5])
        E = groups * max(2, _log(rng, 4, 256) // groups)
        keep = rng.randrange(1, groups + 1)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randrange(1, min(12, keep * (E // groups)) + 1),
                    score=rng.choice(["sigmoid", "softmax", "sqrtsoftplus"]), bias=rng.random() < 0.5, groups=groups,
                    keep=keep, bf16=rng.random() < 0.4)
    if op == "linear":
        T, N, K = _log(rng, 1, 2048), 16 * _log(rng, 1, 512), 32 * _log(rng, 2, 200)
        while T * N * K > 2048 * 4096 * 4096:
            T = max(1, T // 2)
        return dict(op=op, T=T, N=N, K=K)
    T, E, K, I = _log(rng, 1, 4096), _log(rng, 4, 150), 32 * _log(rng, 6, 128), 32 * _log(rng, 3, 48)
    k = rng.randrange(1, min(8, E) + 1)
    while E * K * I > 128 * 4096 * 1024:
        E = max(k, E - E // 4)
    while T * k * K * I > 4096 * 6 * 4096 * 1024:
        T //= 2
    return dict(op=op, T=T, E=E, k=k, K=K, I=I, pad=rng.random() < 0.3)


def _scales(K, group):
    return -(-K // group)


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["D"]
        return {"bytes": n * (2 + 4 * c["residual"] + 2 * c["y"] + c["codes"]) + 2 * c["D"]
                + c["codes"] * c["T"] * _scales(c["D"], 128), "flops": 6 * n}
    if c["op"] == "route":
        n = c["T"] * c["E"]
        return {"bytes": n * (2 if c["bf16"] else 4) + 4 * c["E"] * c["bias"] + 8 * c["T"] * c["k"], "flops": 4 * n}
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": N * (K // 2 + K // 32) + T * (K + _scales(K, 128)) + 2 * T * N, "flops": 2 * T * N * K}
    T, E, k, K, I = c["T"], c["E"], c["k"], c["K"], c["I"]
    read = E * (1 - (1 - k / E) ** T)  # experts that some row chose, at even odds
    return {"bytes": int(read * 3 * I * K * 17 / 32) + T * (K + _scales(K, 128)) + 2 * T * K + 8 * T * k,
            "flops": 6 * T * k * I * K}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _weight(g, *shape):
    """E2M1 codes [.., N, K/2] as a normal distribution's blocks give them, with E8M0 bytes [.., N, K/32] such
    that a row's product with unit activations is of unit size."""
    *lead, K = shape
    # Quantiles of |normal| / (amax / 6) of a block of 32, in 16ths, with a sign.
    mag = torch.tensor([0, 0, 1, 1, 1, 2, 2, 2, 3, 3, 4, 4, 5, 5, 6, 7], device="cuda")
    u = torch.arange(32, device="cuda")
    nib = mag[u % 16] + 8 * (u // 16)
    pair = torch.arange(1024, device="cuda")
    lut = (nib[pair % 32] + 16 * nib[pair // 32]).byte()
    codes = torch.randint(0, 1024, (*lead, K // 2), generator=g, device="cuda", dtype=torch.int32)
    mid = 127 - 1 - int(round(0.5 * math.log2(K)))
    sf = torch.randint(mid - 1, mid + 1, (*lead, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    return lut[codes], sf


def _quant8(y):
    """[.., D] float32 -> E4M3 codes [.., D] and E8M0 bytes [.., ceil(D/128)]: per 128 values the smallest power
    of two 2^e with max |y| <= 448 * 2^e, codes to nearest, ties to the even code."""
    D = y.shape[-1]
    g = torch.nn.functional.pad(y, (0, -D % 128)).unflatten(-1, (-1, 128))
    m, x = torch.frexp(g.abs().amax(-1))
    e = torch.where(m == 0, torch.full_like(x, -127), x - 9 + (m > 0.875).int()).clamp(min=-127)
    v = torch.ldexp(g, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return v.flatten(-2)[..., :D].contiguous(), (e + 127).byte()


def prepare(case, seed):
    s, g = dict(case), _gen(seed)
    if s["op"] == "norm":
        # A residual stream has a few large columns; the branch that is added is smaller.
        T, D = s["T"], s["D"]
        big = 1 + 30 * (torch.rand(D, generator=g, device="cuda") < 0.004)
        s["x"] = (_rand((T, D), g, 0.7) * (1 if s["residual"] else big)).bfloat16()
        s["res"] = (_rand((T, D), g, 2.0) * big).bfloat16() if s["residual"] else None
        s["weight"] = (1 + _rand((D,), g, 0.2)).bfloat16()
        return s
    if s["op"] == "route":
        E = s["E"]
        # Some experts are liked by every token; the bias works against it.
        liked = _rand((E,), g, 0.7)
        s["logits"] = _rand((s["T"], E), g, 1.3) + liked
        if s["bf16"]:
            s["logits"] = s["logits"].bfloat16()
        s["b"] = -0.15 * liked if s["bias"] else None
        return s
    T, K = s["T"], s["K"]
    a, s["a_sf"] = _quant8(_rand((T, K), g))
    s["a"] = a.view(torch.uint8)
    if s["op"] == "linear":
        s["w"], s["w_sf"] = _weight(g, s["N"], K)
        if own:  # once, when the weight is loaded
            import mxfp8_block_scaled_inv_gb300 as mxq

            s["w4"] = mxq.mxq_prepare_w4(s["w"], s["w_sf"])
        return s
    E, I, k = s["E"], s["I"], s["k"]
    s["w13"], s["w13_sf"] = _weight(g, E, 2 * I, K)  # rows [0, I) gate, [I, 2I) up
    s["w2"], s["w2_sf"] = _weight(g, E, K, I)
    top = (_rand((T, E), g) + _rand((E,), g, 0.4)).topk(k, -1)
    s["ids"], s["wt"] = top.indices.int(), 2.5 * top.values.softmax(-1)
    if s["pad"]:  # the batch is padded to a captured size: rows without experts at its end
        s["ids"][T - T // 8:] = -1
    live = s["ids"][s["ids"] >= 0].long()
    s["cap"] = int(torch.bincount(live, minlength=1).max()) if live.numel() else 1
    if own:
        import mxfp8_block_scaled_inv_gb300 as mxq

        s["w13p"] = mxq.mxq_prepare_w4(s["w13"].view(E * 2, I, K // 2), s["w13_sf"].view(E * 2, I, K // 32))
        s["w2p"] = mxq.mxq_prepare_w4(s["w2"], s["w2_sf"])
    return s


# -------------------------------------------------------------- plain forms
def _act(codes, sf):
    K = codes.shape[-1]
    v = codes.view(torch.float8_e4m3fn).float()
    return v * torch.exp2(sf.float() - 127).repeat_interleave(128, -1)[..., :K]


def _wt(codes, sf):
    """The float32 values of E2M1 codes [.., K/2] with scale bytes [.., K/32]."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack([t[(codes & 15).int()], t[(codes >> 4).int()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(sf.float() - 127)[..., None]).flatten(-2)


def _plain_norm(s):
    x = s["x"]
    if s["res"] is not None:
        x = (x.float() + s["res"].float()).bfloat16()
    v = x.float()
    y = (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["weight"].float()).bfloat16()
    codes, sf = _quant8(y.float()) if s["codes"] else (None, None)
    return _norm_outputs(s, x, y, codes, sf)


def _norm_outputs(s, x, y, codes, sf):
    out = {}
    if s["residual"]:
        out["residual"] = x
    if s["y"]:
        out["y"] = y
    if s["codes"]:
        out["codes"], out["scales"] = codes, sf.view(torch.float8_e8m0fnu)
    return out


def _plain_scores(s, logits):
    if s["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    if s["score"] == "softmax":
        p = torch.exp(logits - logits.amax(-1, keepdim=True))
        return p / p.sum(-1, keepdim=True)
    return torch.sqrt(torch.log1p(torch.exp(logits)))


def _plain_route(s):
    T, E, G = s["T"], s["E"], s["groups"]
    p = _plain_scores(s, s["logits"].double())
    c = p + s["b"].double() if s["bias"] else p
    if G > 1:
        in_group = c.view(T, G, E // G)
        best = in_group.sort(-1, descending=True).values[..., :2].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, :s["keep"]]
        see = torch.zeros((T, G), dtype=torch.bool, device=c.device).scatter_(1, kept, True)
        c = in_group.masked_fill(~see[..., None], -math.inf).view(T, E)
    ids = c.sort(dim=-1, descending=True, stable=True).indices[:, :s["k"]]
    w = p.gather(1, ids)
    return ids.int(), (2.5 * w / (w.sum(-1, keepdim=True) + 1e-20)).float()


def _plain_linear(s):
    return torch.matmul(_act(s["a"], s["a_sf"]), _wt(s["w"], s["w_sf"]).t()).bfloat16()


def _plain_mlp(s, x, w13, w2):
    """x [b, n, K] through the experts w13 [b, 2I, K], w2 [b, K, I]."""
    gu = torch.matmul(x, w13.transpose(1, 2))
    g, u = gu[..., :s["I"]], gu[..., s["I"]:]
    h, h_sf = _quant8(g / (1 + torch.exp(-g)) * u)
    return torch.matmul(_act(h, h_sf), w2.transpose(1, 2))


def _plain_experts(s):
    T, E, k, K = s["T"], s["E"], s["k"], s["K"]
    x, ids = _act(s["a"], s["a_sf"]), s["ids"].long().flatten()
    live = ids >= 0
    if T * k <= E:  # a few rows: their experts' weights, row by row
        at = ids.clamp(min=0)
        y = _plain_mlp(s, x.repeat_interleave(k, 0)[:, None], _wt(s["w13"][at], s["w13_sf"][at]),
                       _wt(s["w2"][at], s["w2_sf"][at]))[:, 0]
    else:  # the rows of each expert, padded to the fullest one's number
        key = torch.where(live, ids, torch.full_like(ids, E))
        order = torch.argsort(key, stable=True)
        count = torch.zeros(E + 1, dtype=torch.long, device=x.device).scatter_add_(0, key, torch.ones_like(key))
        rank = torch.arange(T * k, device=x.device) - (count.cumsum(0) - count)[key[order]]
        place = torch.zeros_like(ids)
        place[order] = key[order] * s["cap"] + rank.clamp(max=s["cap"] - 1)
        pad = torch.zeros(((E + 1) * s["cap"], K), device=x.device)
        pad[place] = x.repeat_interleave(k, 0)
        y = _plain_mlp(s, pad[:E * s["cap"]].view(E, s["cap"], K), _wt(s["w13"], s["w13_sf"]),
                       _wt(s["w2"], s["w2_sf"])).view(-1, K)
        y = y[place.clamp(max=E * s["cap"] - 1)]
    y = torch.where(live[:, None], y * s["wt"].flatten()[:, None], torch.zeros_like(y))
    return y.view(T, k, K).sum(1).bfloat16()


def run(state):
    s = state
    if not own:
        return {"norm": _plain_norm, "route": _plain_route, "linear": _plain_linear,
                "experts": _plain_experts}[s["op"]](s)
    import mxfp8_block_scaled_inv_gb300 as mxq

    if s["op"] == "norm":
        x, y, codes, sf = mxq.mxq_add_rms_norm(s["x"], s["weight"], EPS, residual=s["res"], want_y=s["y"],
                                               want_codes=s["codes"])
        return _norm_outputs(s, x, y, None if codes is None else codes.view(torch.float8_e4m3fn), sf)
    if s["op"] == "route":
        return mxq.mxq_route(s["logits"], s["k"], scoring=s["score"], bias=s["b"], groups=s["groups"],
                             topk_groups=s["keep"], group_top=2, renormalise=True, scale=2.5)
    if s["op"] == "linear":
        return mxq.mxq_linear_a8w4(s["a"], s["a_sf"], s["w4"], s["N"])
    return mxq.mxq_experts_a8w4(s["a"], s["a_sf"], s["ids"], s["wt"], s["w13p"], s["w2p"], s["I"])


# ------------------------------------------------------- 64-bit definitions
def _exact8(y):
    """Per 128 values of y [.., D] float64: the values of the nearest E4M3 codes, and the scale."""
    D = y.shape[-1]
    codes, scales = torch.empty_like(y), []
    for a in range(0, D, 128):
        part = y[..., a:a + 128]
        top = part.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)).clamp(min=-127)
        e = torch.where((e > -127) & (top <= 448.0 * torch.exp2(e - 1)), e - 1, e)
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
        v = part * torch.exp2(-e)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        codes[..., a:a + 128] = torch.round(v / step) * step
        scales.append(torch.exp2(e))
    return codes, torch.cat(scales, -1)


def _exact_act(codes, sf):
    v = codes.view(torch.float8_e4m3fn).double()
    for i in range(sf.shape[-1]):
        v[..., 128 * i:128 * i + 128] *= torch.exp2(sf[..., i:i + 1].double() - 127)
    return v


def _exact_wt(codes, sf):
    v = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=torch.float64, device="cuda")
    for half in (0, 1):
        n = (codes >> (4 * half)) & 15
        m, e = (n & 1).double(), ((n >> 1) & 3).double()
        mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e - 1))
        v[..., half::2] = torch.where(n >= 8, -mag, mag)
    return v * torch.exp2(sf.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        x = s["x"].double()
        if s["residual"]:
            # The stored sum is a BF16 number by definition, and the norm is that number's.
            out = x + s["res"].double()
            x = out.float().bfloat16().double()
        else:
            out = x
        y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / s["D"] + EPS) * s["weight"].double()
        r = {}
        if s["residual"]:
            r["residual"] = out
        if s["y"]:
            r["y"] = y
        if s["codes"]:
            # The codes are those of the BF16 form by definition, whether it is stored or not.
            r["codes"], r["scales"] = _exact8(y.float().bfloat16().double())
        return r
    if s["op"] == "route":
        x = s["logits"].double()
        if s["score"] == "sigmoid":
            p = 1 / (1 + torch.exp(-x))
        elif s["score"] == "softmax":
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
        else:
            p = torch.sqrt(torch.log1p(torch.exp(x)))
        c = p.clone() if s["b"] is None else p + s["b"].double()
        G, n, rows = s["groups"], s["E"] // s["groups"], torch.arange(s["T"], device="cuda")
        if G > 1:
            tops = torch.stack([c[:, i * n:(i + 1) * n].topk(2, -1).values.sum(-1) for i in range(G)], -1)
            keep = torch.zeros((s["T"], G), dtype=torch.bool, device="cuda")
            for _ in range(s["keep"]):
                best = tops.argmax(-1)
                keep[rows, best] = True
                tops[rows, best] = -math.inf
            c[~keep.repeat_interleave(n, -1)] = -math.inf
        w = []
        for _ in range(s["k"]):
            i = c.argmax(-1)
            w.append(p[rows, i])
            c[rows, i] = -math.inf
        w = torch.stack(w, -1)
        return None, 2.5 * w / w.sum(-1, keepdim=True)
    a = _exact_act(s["a"], s["a_sf"])
    if s["op"] == "linear":
        return a @ _exact_wt(s["w"], s["w_sf"]).T
    out = torch.zeros((s["T"], s["K"]), dtype=torch.float64, device="cuda")
    for e in range(s["E"]):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        gu = a[t] @ _exact_wt(s["w13"][e], s["w13_sf"][e]).T
        g, u = gu[:, :s["I"]], gu[:, s["I"]:]
        h, sc = _exact8(g * u / (1 + torch.exp(-g)))
        h *= sc.repeat_interleave(128, -1)[:, :s["I"]]
        out.index_add_(0, t, h @ _exact_wt(s["w2"][e], s["w2_sf"][e]).T * s["wt"][t, j].double()[:, None])
    return out
