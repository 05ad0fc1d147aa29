"""Cases that measure the attention operators over this library's KV cache.

Three operators: attention over a paged BF16 / E4M3 cache with a sliding
window and a few first keys that stay visible (``attn``), the same attention
over a cache held in 4 bits (``attn`` with ``cache="e2m1"``), and the insertion
of rotated KV rows into the 4-bit cache (``insert``).  The keys and the values
of a token are one row of the cache, shared by all query heads, as
``mxq_rope_kv_insert`` writes it.

``own`` selects what ``run`` computes: the plain form (elementary torch
operations in 32 bits) or the library's entry points.
"""

import math

import numpy as np
import torch

own = False

GOLDEN = 0.6180339887498949
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One sequence, one new token, 16 heads (a head-sharded server): latency only.
        dict(name="win decode 1x16", op="attn", cache="bf16", B=1, nq=1, H=16, D=512, len=300,
             W=128, S=4, page=64, vary=False),
        # A decode batch of short-window layers over the E4M3 cache.
        dict(name="win decode 64x64 e4m3", op="attn", cache="e4m3", B=64, nq=1, H=64, D=512, len=6000,
             W=1024, S=4, page=64, vary=True),
        # A few long conversations in BF16, wide window.
        dict(name="win decode 16x64 bf16", op="attn", cache="bf16", B=16, nq=1, H=64, D=512, len=30000,
             W=8192, S=16, page=128, vary=True),
        # Ragged chunks of several requests on a small odd-headed model, prefixes cached.
        dict(name="win ragged 7x12", op="attn", cache="e4m3", B=7, nq=301, H=12, D=192, len=2500,
             W=777, S=3, page=16, vary=True),
        # The 8192-token prefill chunk with a narrow window: queries and outputs are the bytes.
        dict(name="win prefill 8192 w128", op="attn", cache="bf16", B=1, nq=8192, H=64, D=512, len=8192,
             W=128, S=4, page=256, vary=False),
        # A chunk at the end of a longer context under a wide window: products are the time.
        dict(name="win prefill 2048 w4096", op="attn", cache="e4m3", B=1, nq=2048, H=64, D=512, len=8192,
             W=4096, S=4, page=64, vary=False),
        # One short request on the 4-bit cache.
        dict(name="kv4 decode 1x16", op="attn", cache="e2m1", B=1, nq=1, H=16, D=512, len=1000,
             W=0, S=0, page=64, vary=False),
        # A decode batch at mixed long contexts, what a 4-bit cache is bought for.
        dict(name="kv4 decode 32x64", op="attn", cache="e2m1", B=32, nq=1, H=64, D=512, len=32768,
             W=0, S=0, page=64, vary=True),
        # One very long context, few rows: the work has to be split along the keys.
        dict(name="kv4 decode 1x64 131072", op="attn", cache="e2m1", B=1, nq=1, H=64, D=512, len=131072,
             W=0, S=0, page=128, vary=False),
        # Chunks of two requests on a smaller head over the 4-bit cache.
        dict(name="kv4 chunks 2x32", op="attn", cache="e2m1", B=2, nq=500, H=32, D=256, len=4001,
             W=0, S=0, page=32, vary=True),
        # The decode step's insertion.
        dict(name="kv4 insert 64", op="insert", T=64, H=64, Dq=512, Dk=512, R=64, slots=4096),
        # The prefill chunk's insertion, query out of place.
        dict(name="kv4 insert 8192", op="insert", T=8192, H=64, Dq=512, Dk=512, R=64, slots=16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "decode4", "decode4", "chunk", "chunk4", "insert"])
    if kind == "insert":
        return dict(op="insert", T=_log(rng, 1, 8000), H=_log(rng, 1, 64), Dq=512, Dk=rng.choice([192, 256, 512, 576]),
                    R=64, slots=16384 + rng.randrange(1000))
    four = kind.endswith("4")
    cache = "e2m1" if four else rng.choice(["bf16", "e4m3"])
    D = rng.choice([64, 128, 192, 256, 320, 512, 512])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if four:
        W, S = 0, 0
    else:
        W, S = rng.choice([0, _log(rng, 16, 8192), _log(rng, 16, 8192)]), rng.choice([0, 1, 4, 17])
        S = S if W else 0
    if kind.startswith("decode"):
        B, L = _log(rng, 1, 128), _log(rng, 1, 40000)
        H, nq = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 4])
        while B * L > 500000:
            L //= 2
    else:
        B, L, H = rng.randrange(1, 6), _log(rng, 20, 8192), _log(rng, 1, 64)
        nq = _log(rng, 2, 2000)
        while B * nq * H * L * D > 3e11:
            nq, H = max(1, nq // 2), max(1, H - H // 4)
    return dict(op="attn", cache=cache, B=B, nq=min(nq, L), H=H, D=D, len=L, W=W, S=S, page=page,
                vary=rng.random() < 0.7)


def _frac(x):
    return x - math.floor(x)


def _lengths(c):
    """(queries, keys) of each sequence; with `vary` they differ, one has no query when there are several."""
    nq, ln = [], []
    for b in range(c["B"]):
        n, l = c["nq"], c["len"]
        if c["vary"] and b > 0:
            l = max(1, int(l * (0.2 + 0.8 * _frac(GOLDEN * b))))
            if c["nq"] > 4:
                n = 0 if b == 3 else 1 if b == 2 else max(1, int(n * _frac(GOLDEN * b + 0.3)))
        nq.append(min(n, l))
        ln.append(l)
    return nq, ln


def work(case):
    c = case
    if c["op"] == "insert":
        T = c["T"]
        rows = T * c["Dk"] * 2 + T * (c["Dk"] // 2 + c["Dk"] // 32) + T * c["Dk"] * 2  # in, held, read back
        return {"bytes": 4 * T * c["H"] * c["Dq"] + rows + T * 16 + 2 * T * c["R"], "flops": 6 * T * c["R"] / 2 * (c["H"] + 1)}
    nq, ln = _lengths(c)
    row = {"bf16": 2 * c["D"], "e4m3": c["D"], "e2m1": c["D"] // 2 + c["D"] // 32}[c["cache"]]
    T, keys, pairs = sum(nq), 0, 0
    for n, l in zip(nq, ln):
        if n == 0:
            continue
        p = np.arange(l - n, l, dtype=np.int64)
        if c["W"]:
            lo = np.maximum(0, p - c["W"] + 1)
            pairs += int((p + 1 - lo + np.minimum(lo, c["S"])).sum())
            keys += int(l - lo[0] + min(lo[0], c["S"]))
        else:
            pairs += int((p + 1).sum())
            keys += l
    return {"bytes": 4 * T * c["H"] * c["D"] + 4 * T * c["H"] + keys * row, "flops": 4.0 * c["D"] * c["H"] * pairs}


# ------------------------------------------------------------------ inputs
def _rand(shape, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * std


def _encode4(y):
    """[n, D] float32 -> (packed E2M1 codes [n, D/2], E8M0 bytes [n, D/32]): per 32 values the smallest
    power of two 2^e with max |y| <= 6 * 2^e, codes to nearest, ties to the even code."""
    n, D = y.shape
    g = y.reshape(n, D // 32, 32)
    m, x = torch.frexp(g.abs().amax(-1))
    e = torch.where(m == 0, torch.full_like(x, -127), x - 3 + (m > 0.75).int()).clamp(-127, 127)
    v = torch.ldexp(g, -e[..., None])
    a = v.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte() + 8 * torch.signbit(v).byte())
    code = code.reshape(n, D // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).byte()


def _decode4(codes, sf):
    """The float32 values that packed codes [..., D/2] with scale bytes [..., D/32] stand for."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack([t[(codes & 15).long()], t[(codes >> 4).long()]], -1).flatten(-2)
    return torch.ldexp(v.unflatten(-1, (-1, 32)), sf.int()[..., None] - 127).flatten(-2)


def prepare(case, seed):
    c, dev = case, "cuda"
    if c["op"] == "insert":
        T, R = c["T"], c["R"]
        g = torch.Generator(device=dev)
        g.manual_seed(seed + 3)
        s = dict(c)
        s["q"] = _rand((T, c["H"], c["Dq"]), seed).bfloat16()
        s["kv"] = _rand((T, c["Dk"]), seed + 1, 4.0).bfloat16()
        s["pos"] = torch.randint(0, 32768, (T,), generator=g, device=dev)
        theta = 10000.0 ** (-2.0 * torch.arange(R // 2, device=dev, dtype=torch.float64) / R)
        ang = torch.arange(32768, device=dev, dtype=torch.float64)[:, None] * theta
        s["cos"], s["sin"] = ang.cos().float().bfloat16(), ang.sin().float().bfloat16()
        s["slot"] = torch.randperm(c["slots"], generator=g, device=dev)[:T]
        s["kv_cache"] = torch.zeros((c["slots"], c["Dk"] // 2), dtype=torch.uint8, device=dev)
        s["kv_sf"] = torch.zeros((c["slots"], c["Dk"] // 32), dtype=torch.uint8, device=dev)
        return s
    nq, ln = _lengths(c)
    T, D, page = sum(nq), c["D"], c["page"]
    pages = -(-max(ln) // page)
    g = torch.Generator(device=dev)
    g.manual_seed(seed + 3)
    total = c["B"] * pages
    bt = torch.randperm(total, generator=g, device=dev).int().reshape(c["B"], pages)
    # Keys of unit size; queries lean towards a direction that the first keys of each sequence share, as
    # trained models' do, so that the first keys draw much of the weight.
    u = _rand((D,), seed + 4)
    q = (_rand((T, c["H"], D), seed) + 0.7 * u).bfloat16()
    kv = _rand((total * page, D), seed + 1)
    first = bt[:, 0].long() * page
    kv[first] += 0.3 * u
    s = dict(c, q=q, bt=bt, nq_max=max(nq), len_max=max(ln), scale=None, sf=None)
    s["q_start"] = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32, device=dev)
    s["lens"] = torch.tensor(ln, dtype=torch.int32, device=dev)
    if c["cache"] == "bf16":
        s["kv"] = kv.bfloat16()
    elif c["cache"] == "e4m3":
        s["scale"] = torch.full((1,), 0.0371, device=dev)
        s["kv"] = (kv / 0.0371).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["kv"], s["sf"] = _encode4(kv)
    return s


# -------------------------------------------------------------- plain forms
def _rotate(x, c, s, R):
    """x [..., D] float32: the pairs (D-R+i, D-R/2+i) rotated by +angle; c, s [..., R/2] float32."""
    D = x.shape[-1]
    x0, x1 = x[..., D - R:D - R // 2], x[..., D - R // 2:]
    return torch.cat([x[..., :D - R], x0 * c - x1 * s, x1 * c + x0 * s], -1)


def _plain_insert(s):
    R = s["R"]
    c, n = s["cos"][s["pos"]].float(), s["sin"][s["pos"]].float()
    q = _rotate(s["q"].float(), c[:, None], n[:, None], R).bfloat16()
    codes, sf = _encode4(_rotate(s["kv"].float(), c, n, R))
    s["kv_cache"][s["slot"]] = codes
    s["kv_sf"][s["slot"]] = sf
    return q, _decode4(s["kv_cache"][s["slot"]], s["kv_sf"][s["slot"]]).bfloat16()


def _plain_attn(s):
    q, bt, page, T = s["q"], s["bt"], s["page"], s["q"].shape[0]
    B, H, D, N, L = s["B"], s["H"], s["D"], s["nq_max"], s["len_max"]
    dev = q.device
    j = torch.arange(L, device=dev)
    slot = bt[:, j // page].long() * page + j % page
    if s["cache"] == "bf16":
        k = s["kv"][slot].float()
    elif s["cache"] == "e4m3":
        k = s["kv"][slot].view(torch.float8_e4m3fn).float() * s["scale"]
    else:
        k = _decode4(s["kv"][slot], s["sf"][slot])
    start = s["q_start"].long()
    nq = start[1:] - start[:-1]
    i = torch.arange(N, device=dev)
    qp = q[(start[:-1, None] + i).clamp(max=T - 1)].float().reshape(B, N * H, D)
    p = (s["lens"].long() - nq)[:, None] + i  # position of each query
    see = j <= p[..., None]
    if s["W"]:
        see &= (j > p[..., None] - s["W"]) | (j < s["S"])
    see &= (i < nq[:, None])[..., None]
    w = torch.matmul(qp, k.transpose(1, 2)).reshape(B, N, H, L)
    w.mul_(D ** -0.5).masked_fill_(~see[:, :, None], -math.inf)
    m = w.amax(-1, keepdim=True).clamp(min=-3e38)
    w.sub_(m).exp_()
    l = w.sum(-1, keepdim=True)
    o = torch.matmul(w.reshape(B, N * H, L), k).reshape(B, N, H, D) / l.clamp(min=1e-30)
    lse = (m + l.log())[..., 0]
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    at = t - start[b]
    return o[b, at].bfloat16(), lse[b, at]


def run(state):
    s = state
    if not own:
        return _plain_insert(s) if s["op"] == "insert" else _plain_attn(s)
    import mxfp8_block_scaled_inv_gb300 as mxq

    if s["op"] == "insert":
        q = mxq.mxq_rope_kv4_insert(s["q"], s["kv"], s["pos"], s["cos"], s["sin"], s["R"], s["slot"],
                                    s["kv_cache"], s["kv_sf"])
        return q, mxq.mxq_kv4_gather(s["kv_cache"], s["kv_sf"], s["slot"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    out = mxq.mxq_attn(s["q"], s["kv"], s["bt"], s["lens"], q_start=s["q_start"], page_size=s["page"],
                       window=s["W"], sinks=s["S"], kv_scale=s["scale"], cache_sf=s["sf"], lse=lse)
    return out, lse


# ------------------------------------------------------- 64-bit definitions
def _exact_rows(s, slots):
    rows = s["kv"][slots]
    if s["cache"] == "bf16":
        return rows.double()
    if s["cache"] == "e4m3":
        return rows.view(torch.float8_e4m3fn).double() * s["scale"].double()
    mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    out = torch.empty((rows.shape[0], rows.shape[1] * 2), dtype=torch.float64, device="cuda")
    for half in (0, 1):
        n = (rows >> (4 * half)) & 15
        out[:, half::2] = mag[(n & 7).long()] * (1.0 - 2.0 * (n >> 3).double())
    return out * torch.exp2(s["sf"][slots].double() - 127.0).repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "insert":
        def turn(x):
            D, R = x.shape[-1], s["R"]
            c, n = s["cos"][s["pos"]].double(), s["sin"][s["pos"]].double()
            while c.dim() < x.dim():
                c, n = c.unsqueeze(1), n.unsqueeze(1)
            a, b = x[..., D - R:D - R // 2].double(), x[..., D - R // 2:].double()
            y = x.double()
            # The rotated values are float32 numbers by definition (the products are exact there).
            y[..., D - R:D - R // 2] = (a * c - b * n).float().double()
            y[..., D - R // 2:] = (b * c + a * n).float().double()
            return y

        y = turn(s["kv"]).reshape(s["T"], -1, 32)
        top = y.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2((top / 6.0).clamp(min=2.0 ** -127))).clamp(-127, 127)
        e = torch.where(top <= 6.0 * torch.exp2(e - 1), e - 1, e)
        v = y * torch.exp2(-e)
        mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        # Nearest of the eight magnitudes; of two equally near ones the even code: odd codes lose ties.
        d = (v.abs()[..., None] - mag).abs() + (torch.arange(8, device="cuda") % 2) * 1e-12
        r = mag[d.argmin(-1)] * torch.where(v < 0, -1.0, 1.0) * torch.exp2(e)
        return turn(s["q"]), r.reshape(s["T"], -1)
    nq, ln = _lengths(case)
    T, H, D, W, S, page = s["q"].shape[0], s["H"], s["D"], s["W"], s["S"], s["page"]
    out = torch.zeros((T, H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, l) in enumerate(zip(nq, ln)):
        step = max(1, min(64, int(4e8 // (H * min(l, W + S + 64 if W else l)))))
        for a in range(0, n, step):
            z = min(n, a + step)
            p = torch.arange(l - n + a, l - n + z, device="cuda")
            lo = max(0, l - n + a - W + 1) if W else 0
            at = torch.cat([torch.arange(0, min(S if W else 0, lo), device="cuda"),
                            torch.arange(lo, l - n + z, device="cuda")])
            k = _exact_rows(s, s["bt"][b, at // page].long() * page + at % page)
            x = torch.einsum("thd,jd->thj", s["q"][t0 + a:t0 + z].double(), k) / math.sqrt(D)
            see = at[None, :] <= p[:, None]
            if W:
                see &= (p[:, None] - at[None, :] < W) | (at[None, :] < S)
            x = torch.where(see[:, None], x, torch.full_like(x, -math.inf))
            lse[t0 + a:t0 + z] = torch.logsumexp(x, -1)
            out[t0 + a:t0 + z] = torch.einsum("thj,jd->thd", torch.exp(x - lse[t0 + a:t0 + z, :, None]), k)
        t0 += n
    return out, lse
