"""What is measured of the few-row operators: the RMS norm that opens a block (dq_rmsnorm_forward) and
the product of few rows with a packed 4-bit weight (dq_rows_forward).

`own` chooses between the plain forms below, elementary torch operations in 32 bits, and the calls a
user makes of the library.  Shapes and inputs follow the repository's own layers (5120 channels, a
13824-wide feed-forward block, low-rank factors of rank 32, 21 frames of 30 x 52 tokens) and generic
ones around them; inputs are synthetic with outlier channels, as the layers' own inputs are.
"""
import math
import struct

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def _norm(name, rows, c, out, residual=True, pad=0, gamma=True):
    return {"name": name, "op": "norm", "rows": rows, "c": c, "out": out, "residual": residual, "pad": pad,
            "gamma": gamma}


def _rows(name, rows, ci, co, x="bf16", rank=32, gelu=False, bias=True, pad=0):
    return {"name": name, "op": "rows", "rows": rows, "ci": ci, "co": co, "x": x, "rank": rank, "gelu": gelu,
            "bias": bias, "pad": pad}


def listed():
    return [
        # one conditioning token before an 8-bit product: latency
        _norm("norm_1x5120_fp8", 1, 5120, "e4m3_token"),
        # an odd width in a wider buffer, no residual: the unaligned path
        _norm("norm_77x1337_bf16", 77, 1337, "bf16", residual=False, pad=6),
        # one frame of 30 x 52 tokens, 8 bits with one scale for each 64 channels
        _norm("norm_1560x5120_fp8g64", 1560, 5120, "e4m3_group64"),
        # all 21 frames before a 4-bit layer, BF16 out
        _norm("norm_32760x5120_bf16", 32760, 5120, "bf16"),
        # the smallest layer
        _rows("rows_1_256to256", 1, 256, 256, rank=16),
        # a conditioning projection of one token
        _rows("rows_1_5120to5120", 1, 5120, 5120),
        # one token through the feed-forward block's first layer, 8-bit input, GELU
        _rows("rows_1_5120to13824_fp8_gelu", 1, 5120, 13824, x="e4m3_token", gelu=True),
        # a small batch through its second layer
        _rows("rows_4_13824to5120", 4, 13824, 5120),
        # one token for each of 21 frames
        _rows("rows_21_5120to13824_gelu", 21, 5120, 13824, gelu=True),
        # a short prompt with 8-bit input in groups of 64, a higher rank, odd count
        _rows("rows_77_2048to5120_fp8g64", 77, 2048, 5120, x="e4m3_group64", rank=128, bias=False),
        # a prompt's keys or values: the longest
        _rows("rows_512_5120to5120", 512, 5120, 5120, pad=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        c = _log(rng, 64, 13824)
        if rng.random() < 0.6:
            c = max(64, c // 64 * 64)
        rows = min(_log(rng, 1, 32760), 32760 * 5120 // c)
        case = _norm("", rows, c, rng.choice(["bf16", "e4m3_token", "e4m3_group64"]), rng.random() < 0.7,
                     rng.choice([0, 0, 1, 8, 24]), rng.random() < 0.8)
    else:
        ci, co = 256 * _log(rng, 1, 54), 256 * _log(rng, 1, 54)
        while ci * co > 5120 * 13824:
            ci, co = 256 * _log(rng, 1, 54), 256 * _log(rng, 1, 54)
        rows = min(_log(rng, 1, 512), 512 * 5120 * 5120 // (ci * co))
        case = _rows("", rows, ci, co, rng.choice(["bf16", "bf16", "e4m3_token", "e4m3_group64"]),
                     16 * rng.randint(1, 8), rng.random() < 0.4, rng.random() < 0.6, rng.choice([0, 0, 64]))
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _cuda_gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, rows, c, pad, outliers=0.01, factor=50.0):
    """BF16 rows with a scale for each channel and a few outlier channels, in a buffer pad wider."""
    buf = torch.zeros(rows, c + pad, dtype=torch.bfloat16, device="cuda")
    s = torch.exp(torch.randn(c, generator=g, device="cuda") * 0.5)
    s = torch.where(torch.rand(c, generator=g, device="cuda") < outliers, s * factor, s)
    for r0 in range(0, rows, 8192):
        n = min(8192, rows - r0)
        buf[r0:r0 + n, :c] = (torch.randn(n, c, generator=g, device="cuda") * s).bfloat16()
    return buf[:, :c]


def _weight(g, co, ci, rank, bias):
    """A packed weight as the packer writes it (include/deltaquant.h), of a random residual, and its factors."""
    r = torch.randn(co, ci, generator=g, device="cuda") * ci ** -0.5
    s_w = float(r.abs().max()) / 2688.0
    sb = (r.reshape(co, ci // 16, 16).abs().amax(2) / (6.0 * s_w)).to(torch.float8_e4m3fn)
    z = r.reshape(co, ci // 16, 16) / (sb.float()[:, :, None] * s_w)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    q = torch.bucketize(z.abs(), edges).to(torch.uint8) | ((z < 0).to(torch.uint8) << 3)
    dqw = (torch.tensor(E2M1, device="cuda")[(q & 7).long()] * torch.where(q > 7, -1.0, 1.0)
           * sb.float()[:, :, None]).bfloat16().reshape(co, ci)
    q = q.reshape(co, ci)
    codes = q[:, 0::2] | (q[:, 1::2] << 4)
    # scales: row = 256 t + 128 h + 32 c + 8 a + i in lane 8 a + i, copied to the four lane quadrants
    s8 = sb.view(torch.uint8).reshape(co // 256, 2, 4, 4, 8, ci // 64, 4)        # t h c a i kb blk
    s8 = s8.permute(0, 5, 3, 1, 4, 2, 6).reshape(co // 256, ci // 64, 1, 1024)   # t kb a h i c blk
    s8 = s8.expand(-1, -1, 4, -1).reshape(-1)
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    off_codes = 256
    off_scales = up(off_codes + co * ci // 2)
    off_dqw = up(off_scales + s8.numel())
    off_bias = up(off_dqw + co * ci * 2)
    total = up(off_bias + co * 4)
    slab = -(-2 * rank // 64) * 64
    head = struct.pack("<IIiiiifIQQQQQ", 0x31575144, 3, co, ci, rank, slab, s_w, int(bias), off_codes, off_scales,
                       off_dqw, total, off_bias)
    blob = torch.zeros(total, dtype=torch.uint8, device="cuda")
    blob[:len(head)] = torch.frombuffer(bytearray(head), dtype=torch.uint8).cuda()
    blob[off_codes:off_codes + co * ci // 2] = codes.reshape(-1)
    blob[off_scales:off_scales + s8.numel()] = s8
    blob[off_dqw:off_dqw + co * ci * 2] = dqw.view(torch.uint8).reshape(-1)
    b = torch.randn(co, generator=g, device="cuda").bfloat16().float() if bias else torch.zeros(co, device="cuda")
    blob[off_bias:off_bias + 4 * co] = b.view(torch.uint8)
    l1 = (torch.randn(rank, ci, generator=g, device="cuda") * ci ** -0.5).bfloat16()
    l2 = (torch.randn(co, rank, generator=g, device="cuda") * rank ** -0.5).bfloat16()
    l2_slab = torch.zeros(co, slab, dtype=torch.bfloat16, device="cuda")
    l2_slab[:, :rank] = l2
    l2_slab[:, rank:2 * rank] = l2
    s_w = struct.unpack("<f", struct.pack("<f", s_w))[0]
    return {"packed": blob, "l1": l1, "l2": l2_slab, "s_w": s_w,
            "codes": blob[off_codes:off_codes + co * ci // 2].view(co, ci // 2),
            "scales": blob[off_scales:off_scales + s8.numel()], "bias": blob[off_bias:off_bias + 4 * co].view(torch.float32)}


def prepare(case, seed):
    g = _cuda_gen(seed)
    if case["op"] == "norm":
        rows, c, pad = case["rows"], case["c"], case["pad"]
        st = {"case": case, "x": _activations(g, rows, c, pad, 0.0), "eps": 1e-6, "residual": None, "gamma": None}
        if case["residual"]:
            st["residual"] = _activations(g, rows, c, pad)
            st["sum"] = torch.zeros(rows, c, dtype=torch.bfloat16, device="cuda")
        if case["gamma"]:
            st["gamma"] = (1.0 + 0.2 * torch.randn(c, generator=g, device="cuda")).bfloat16()
        if case["out"] == "bf16":
            st["y"] = torch.zeros(rows, c, dtype=torch.bfloat16, device="cuda")
        else:
            st["y"] = torch.zeros(rows, c, dtype=torch.float8_e4m3fn, device="cuda")
            groups = 1 if case["out"] == "e4m3_token" else -(-c // 64)
            st["scales"] = torch.zeros(rows, groups, device="cuda")
        return st
    rows, ci, co = case["rows"], case["ci"], case["co"]
    st = {"case": case, **_weight(g, co, ci, case["rank"], case["bias"])}
    x = _activations(g, rows, ci, case["pad"])
    st["x_scales"] = None
    if case["x"] != "bf16":   # rows quantised before: codes and their scales
        n = ci if case["x"] == "e4m3_token" else 64
        v = x.float().reshape(rows, ci // n, n)
        s = v.abs().amax(2) / 448.0
        x = (v / s[:, :, None]).to(torch.float8_e4m3fn).reshape(rows, ci)
        st["x_scales"] = s.contiguous()
    st["x"] = x
    st["y"] = torch.zeros(rows, co, dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return (_run_norm if st["case"]["op"] == "norm" else _run_rows)(st)


def _run_norm(st):
    c, out = st["case"]["c"], st["case"]["out"]
    res, gamma = st["residual"], st["gamma"]
    if own:
        import video_diffusion_w4a4_b200 as dq
        fmt = {"bf16": dq.DQ_ROWS_BF16, "e4m3_token": dq.DQ_ROWS_E4M3, "e4m3_group64": dq.DQ_ROWS_E4M3_GROUP64}[out]
        x = st["x"]
        dq.dq_rmsnorm_forward(x, x.shape[0], c, st["y"], x_stride=x.stride(0), residual=res,
                              residual_stride=res.stride(0) if res is not None else 0, sum_out=st.get("sum"),
                              gamma=gamma, eps=st["eps"], y_format=fmt, y_scales=st.get("scales"))
        return {k: st[k] for k in ("y", "scales", "sum") if k in st}
    h = st["x"].float()
    if res is not None:
        h = h + res.float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + st["eps"])
    if gamma is not None:
        y = y * gamma.float()
    got = {} if res is None else {"sum": h.bfloat16()}
    if out == "bf16":
        return {**got, "y": y.bfloat16()}
    n = c if out == "e4m3_token" else 64
    rows, fill = y.shape[0], -c % n
    if fill:
        y = torch.cat([y, y.new_zeros(rows, fill)], 1)
    y = y.view(rows, -1, n)
    s = y.abs().amax(2) / 448.0
    q = torch.where(s[:, :, None] > 0, y / s[:, :, None], 0.0).clamp(-448.0, 448.0)
    return {**got, "y": q.reshape(rows, -1)[:, :c].to(torch.float8_e4m3fn), "scales": s}


def _run_rows(st):
    case, x = st["case"], st["x"]
    rows, ci, co, rank = case["rows"], case["ci"], case["co"], case["rank"]
    if own:
        import video_diffusion_w4a4_b200 as dq
        if "workspace" not in st:   # a user's program keeps it from call to call
            st["workspace_bytes"] = dq.dq_rows_workspace_bytes(rows, ci, co, rank)
            st["workspace"] = torch.zeros(st["workspace_bytes"], dtype=torch.uint8, device="cuda")
        fmt = {"bf16": dq.DQ_ROWS_BF16, "e4m3_token": dq.DQ_ROWS_E4M3, "e4m3_group64": dq.DQ_ROWS_E4M3_GROUP64}
        dq.dq_rows_forward(x, rows, ci, co, rank, st["packed"], st["l1"], st["l2"], st["y"], st["workspace"],
                           st["workspace_bytes"], x_stride=x.stride(0), x_format=fmt[case["x"]],
                           x_scales=st["x_scales"],
                           epilogue=dq.DQ_EPILOGUE_GELU if case["gelu"] else dq.DQ_EPILOGUE_NONE)
        return st["y"]
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    codes = torch.stack([st["codes"] & 15, st["codes"] >> 4], 2).view(co, ci // 16, 16)
    sb = st["scales"].view(co // 256, ci // 64, 4, 4, 2, 8, 4, 4)[:, :, 0]        # t kb a h i c blk
    sb = sb.permute(0, 3, 5, 2, 4, 1, 6).reshape(co, ci // 16).view(torch.float8_e4m3fn).float()
    w = (lut[codes.int()] * sb[:, :, None]).view(co, ci)
    v = x.float()
    if st["x_scales"] is not None:
        v = (v.view(rows, st["x_scales"].shape[1], -1) * st["x_scales"][:, :, None]).view(rows, ci)
    y = (v @ w.t()) * st["s_w"] + (v @ st["l1"].float().t()) @ st["l2"][:, :rank].float().t() + st["bias"]
    if case["gelu"]:
        y = 0.5 * y * (1.0 + torch.erf(y * 0.7071067811865476))
    return y.bfloat16()


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["c"]
        groups = case["rows"] * (1 if case["out"] == "e4m3_token" else -(-case["c"] // 64))
        b = 2 * n + (4 * n if case["residual"] else 0) + (2 * case["c"] if case["gamma"] else 0)
        b += 2 * n if case["out"] == "bf16" else n + 4 * groups
        return {"bytes": b, "flops": 6 * n}
    m, ci, co, r = case["rows"], case["ci"], case["co"], case["rank"]
    b = co * ci // 2 + co * ci // 16 + 2 * r * (ci + co) + (4 * co if case["bias"] else 0) + 2 * m * co
    if case["x"] == "bf16":
        b += 2 * m * ci
    else:
        b += m * ci + 4 * m * (1 if case["x"] == "e4m3_token" else ci // 64)
    return {"bytes": b, "flops": 2 * m * (ci * co + r * (ci + co))}


# ------------------------------------------------------------------ the definitions in 64 bits

def _e4m3_nearest(v):
    """v rounded to E4M3 (nearest, ties to even, saturating), in 64 bits."""
    a = v.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a))))
    e = torch.where(torch.ldexp(torch.ones_like(a), e) > a, e - 1, e)
    e = torch.where(torch.ldexp(torch.ones_like(a), e + 1) <= a, e + 1, e).clamp(min=-6)
    step = torch.ldexp(torch.ones_like(a), e - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448.0)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        h = st["x"].double()
        if st["residual"] is not None:
            h = h + st["residual"].double()
        rows, c = h.shape
        y = h / torch.sqrt((h * h).sum(1) / c + st["eps"])[:, None]
        if st["gamma"] is not None:
            y = y * st["gamma"].double()
        got = {} if st["residual"] is None else {"sum": h}
        if case["out"] == "bf16":
            return {**got, "y": y}
        q, scales = torch.empty_like(y), []
        n = c if case["out"] == "e4m3_token" else 64
        for j in range(0, c, n):
            part = y[:, j:j + n]
            s = part.abs().max(1).values / 448.0
            q[:, j:j + n] = _e4m3_nearest(part / torch.where(s > 0, s, torch.ones_like(s))[:, None])
            scales.append(s)
        return {**got, "y": q, "scales": torch.stack(scales, 1)}
    m, ci, co, r = case["rows"], case["ci"], case["co"], case["rank"]
    v = st["x"].double()
    if case["x"] != "bf16":
        v = v * torch.repeat_interleave(st["x_scales"].double(), ci // st["x_scales"].shape[1], 1)
    y = (v @ st["l1"].double().t()) @ st["l2"][:, :r].double().t() + st["bias"].double()
    # the scale of 16-channel block b of weight row o sits at the byte the layout's formula gives
    o, b = torch.arange(co, device="cuda")[:, None], torch.arange(ci // 16, device="cuda")[None]
    n = o % 256
    byte = 4 * (4 * (n // 128) + (n % 128) // 32) + b % 4
    at = ((o // 256) * (ci // 64) + b // 4) * 4096 + (n % 32 // 8) * 256 + (byte // 16) * 128 + (n % 8) * 16 + byte % 16
    sb = st["scales"][at].long()
    sb = torch.where(sb >= 8, torch.ldexp(1.0 + (sb % 8).double() / 8, sb // 8 - 7), (sb % 8).double() / 512)
    for k in range(2):   # the channels of the low nibbles, then those of the high ones
        q = (st["codes"] >> (4 * k)).long()
        e, f = q // 2 % 4, (q % 2).double()
        w = torch.where(e > 0, torch.ldexp(1.0 + f / 2, e - 1), f / 2) * (1 - 2 * (q // 8 % 2)).double()
        w = (w.view(co, ci // 16, 8) * sb[:, :, None]).view(co, ci // 2)
        y += v[:, k::2] @ w.t() * st["s_w"]
        del q, e, f, w
    if case["gelu"]:
        y = y * 0.5 * torch.special.erfc(-y / math.sqrt(2.0))
    return y
