"""Cases of the products in microscaled 4-bit floating point: activations to 4 bits and back, the shared projection, the
experts' products, in plain form (`own` false) and as the library's calls (`own` true).

Formats: "nvfp4" has one E4M3 scale for each 16 neighbours of a row and an FP32 scale over all, "mxfp4" a power of two for
each 32.  Elements are E2M1 codes, two in a byte, the even one in the low half."""

import math

import torch

own = False

DEV = "cuda"
BLOCK = {"nvfp4": 16, "mxfp4": 32}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decoded token's activations before its experts
        dict(name="quantize T1", op="quantize", T=1, K=6144, format="nvfp4", globals=True),
        # an odd verify batch between the experts' two products
        dict(name="quantize T300 mx", op="quantize", T=300, K=2048, format="mxfp4", globals=False),
        # a prefill batch
        dict(name="quantize T8192", op="quantize", T=8192, K=6144, format="nvfp4", globals=True),
        # the shared expert of one decoded token, gate and up; latency counts
        dict(name="linear T1", op="linear", T=1, K=6144, N=4096, format="nvfp4", act="swiglu"),
        # the shared expert of a decode batch, down
        dict(name="linear T64 mx", op="linear", T=64, K=2048, N=6144, format="mxfp4", act="none"),
        # the shared expert of a prefill batch, gate and up
        dict(name="linear T4096", op="linear", T=4096, K=6144, N=4096, format="nvfp4", act="swiglu"),
        # one decoded token: 8 experts' gate and up weights
        dict(name="experts T1", op="experts", T=1, E=64, k=8, K=6144, N=4096, format="nvfp4", act="swiglu", gather=True, skew=0.0),
        # a decode batch: nearly every expert is read for one to a few rows
        dict(name="experts T64", op="experts", T=64, E=256, k=8, K=6144, N=4096, format="nvfp4", act="swiglu", gather=True, skew=0.5),
        # a prefill batch, uneven experts: the largest product
        dict(name="experts T8192", op="experts", T=8192, E=256, k=8, K=6144, N=4096, format="nvfp4", act="swiglu", gather=True,
             skew=0.5),
        # an odd verify batch of a ragged layer: down projection of rows that lie expert after expert
        dict(name="experts T37 ragged", op="experts", T=37, E=168, k=6, K=1088, N=2056, format="nvfp4", act="none", gather=False,
             skew=0.5),
        # a middle batch's down projection with powers of two as scales
        dict(name="experts T2048 mx", op="experts", T=2048, E=256, k=8, K=2048, N=6144, format="mxfp4", act="none", gather=False,
             skew=0.5),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step * step, max(-(-lo // step) * step, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "linear", "experts", "experts"])
    format = rng.choice(["nvfp4", "nvfp4", "mxfp4"])
    step = 64 if format == "nvfp4" else 128
    if op == "quantize":
        return dict(op=op, T=_log(rng, 1, 8192), K=_log(rng, 256, 6144, step), format=format,
                    globals=format == "nvfp4" and rng.random() < 0.5)
    act = rng.choice(["none", "swiglu"])
    K = _log(rng, 256, 6144 if act == "swiglu" else 2048, step)  # gate and up, or down
    N = _log(rng, 128, 2048, 8) * 2 if act == "swiglu" else _log(rng, 256, 6144, 8)
    if op == "linear":
        return dict(op=op, T=_log(rng, 1, 4096), K=K, N=N, format=format, act=act)
    return dict(op=op, T=_log(rng, 1, 8192), E=_log(rng, 8, 256), k=rng.randint(1, 8), K=K, N=N, format=format, act=act,
                gather=rng.random() < 0.5, skew=rng.choice([0.0, 0.5]))


def _four_bits(x, format, g=None):
    """x [.., K] as E2M1 codes, one in a byte, and scale bytes [.., K / block]: the quotients and their roundings in 64 bits."""
    b = x.double().reshape(*x.shape[:-1], -1, BLOCK[format])
    amax = b.abs().amax(-1, keepdim=True)
    if format == "nvfp4":
        unit = 1.0 if g is None else g.double()
        q = amax / (6.0 * unit)
        step = torch.ldexp(torch.ones_like(q), torch.frexp(q).exponent.clamp(min=-5) - 4)  # of E4M3 at q
        s = (torch.round(q / step) * step).clamp(max=448.0)
        byte = s[..., 0].float().to(torch.float8_e4m3fn).view(torch.uint8)
        s = s * unit
    else:
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(min=-127)
        byte = (e[..., 0] + 127).to(torch.uint8)
        s = torch.ldexp(torch.ones_like(amax), e)
    v = torch.where(s > 0, b.abs() / torch.where(s > 0, s, 1.0), 0.0)
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    v = (torch.round(v / step) * step).clamp(max=6.0)
    code = torch.where(v <= 2, 2 * v, torch.where(v <= 4, v + 2, 7.0)).to(torch.uint8)
    return (code | (torch.signbit(b).to(torch.uint8) << 3)).reshape(x.shape), byte


def _packed(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _ids(c, g):
    """k distinct experts a token, some experts more popular than others."""
    T, E, k = c["T"], c["E"], c["k"]
    popular = torch.randn(E, generator=g, device=DEV) * c["skew"]
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    return torch.topk(popular + noise, k, dim=1).indices.to(torch.int32)


def _bf16(g, std, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16) * std


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case=c)
    T, K, format = c["T"], c["K"], c["format"]
    if c["op"] == "quantize":
        # activations: a few channels are far larger than the rest
        s["x"] = _bf16(g, 1.0, T, K) * torch.exp(torch.randn(K, generator=g, device=DEV)).bfloat16()
        s["g"] = s["x"].abs().amax().float().reshape(1) / (448.0 * 6.0) if c["globals"] else None
        return s
    E = c.get("E", 1)
    n = T if c["op"] == "linear" else T * c["k"]
    # weights in 4 bits: a few experts at a time
    parts = []
    s["factor"] = torch.empty(E, device=DEV)
    each = max(1, 2**28 // (c["N"] * K))
    for i in range(0, E, each):
        w = _bf16(g, 0.02, min(each, E - i), c["N"], K)
        gw = (w.abs().amax() / (448.0 * 6.0)).float() if format == "nvfp4" else None
        code, byte = _four_bits(w, format, gw)
        parts.append((_packed(code), byte))
        s["factor"][i:i + each] = 1.0 if gw is None else gw
        del w, code
    s["w"], s["w_scales"] = (torch.cat(v) for v in zip(*parts))
    if c["op"] == "experts":
        ids = _ids(c, g)
        order = torch.argsort(ids.reshape(-1), stable=True)
        s["counts"] = torch.bincount(ids.reshape(-1), minlength=E).to(torch.int32)
        s["offsets"] = torch.cat([s["counts"].new_zeros(1), torch.cumsum(s["counts"], 0, dtype=torch.int32)])
        s["row_token"] = (order // c["k"]).to(torch.int32) if c["gather"] else None
        s["expert"] = ids.reshape(-1)[order].to(torch.int64)
        s["widest"] = int(s["counts"].max().item())
    x = _bf16(g, 1.0, T if c["op"] == "linear" or c["gather"] else n, K)
    gx = x.abs().amax().float() / (448.0 * 6.0) if format == "nvfp4" else None
    code, s["x_scales"] = _four_bits(x, format, gx)
    s["x"] = _packed(code)
    if gx is not None:
        s["factor"] *= gx
    if own:  # the scales of the weights in the products' own order, made once with the weights
        import moe_decode_layer_logits_gb300 as M

        if c["op"] == "linear":
            s["w"], s["w_scales"] = s["w"][0], s["w_scales"][0]
        s["w_scales"] = M.moe_fp4_weight_scales(s["w_scales"], format=format, act=None if c["act"] == "none" else c["act"])
    return s


# ------------------------------------------------------------------ plain forms


def _scale_values(byte, format):
    if format == "nvfp4":
        return byte.view(torch.float8_e4m3fn).float()
    return torch.exp2(byte.float() - 127.0)


def _pairs():
    """The two values of each byte."""
    one = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=DEV)
    return torch.stack([one.repeat(16), one.repeat_interleave(16)], dim=1)


def _values(packed, byte, format):
    """What codes and scales stand for, without the scale over all: FP32, exact."""
    v = torch.index_select(_pairs(), 0, packed.reshape(-1).to(torch.int32))
    v = v.reshape(*byte.shape, BLOCK[format])
    v.mul_(_scale_values(byte, format)[..., None])
    return v.reshape(*packed.shape[:-1], -1)


def _quantize_plain(s, c):
    code, byte = _four_bits(s["x"], c["format"], s["g"])
    v = _values(_packed(code), byte, c["format"])
    return (v if s["g"] is None else v.double() * s["g"].double()).to(torch.bfloat16)


def _act_plain(y, act):
    if act == "none":
        return y.to(torch.bfloat16)
    gate, up = y.chunk(2, dim=-1)
    return (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)


def _linear_plain(s, c):
    y = _values(s["x"], s["x_scales"], c["format"]) @ _values(s["w"][0], s["w_scales"][0], c["format"]).T
    return _act_plain(y * s["factor"], c["act"])


def _experts_plain(s, c):
    x = _values(s["x"], s["x_scales"], c["format"])
    if s["row_token"] is not None:
        x = x[s["row_token"].long()]
    e = s["expert"]
    if len(e) * 4 <= c["E"]:  # few rows: each row's own weights
        w = _values(s["w"][e], s["w_scales"][e], c["format"])
        return _act_plain((w @ x[:, :, None])[:, :, 0] * s["factor"][e, None], c["act"])
    at = torch.arange(len(e), device=e.device) - s["offsets"][e].long()
    padded = torch.zeros(c["E"], s["widest"], c["K"], device=x.device)
    padded[e, at] = x
    y = torch.bmm(padded, _values(s["w"], s["w_scales"], c["format"]).transpose(1, 2))[e, at]
    return _act_plain(y * s["factor"][e, None], c["act"])


def run(state):
    s, c = state, state["case"]
    if own:
        import moe_decode_layer_logits_gb300 as M

        if c["op"] == "quantize":
            codes, scales = M.moe_fp4_quantize(s["x"], format=c["format"], global_scale=s["g"])
            return M.moe_fp4_dequantize(codes, scales, format=c["format"], global_scale=s["g"])
        act = None if c["act"] == "none" else c["act"]
        if c["op"] == "linear":
            return M.moe_fp4_linear(s["x"], s["x_scales"], s["w"], s["w_scales"], format=c["format"], factor=s["factor"], act=act)
        return M.moe_fp4_expert_linear(s["x"], s["x_scales"], s["w"], s["w_scales"], s["offsets"], s["counts"],
                                       format=c["format"], factor=s["factor"], row_token=s["row_token"], act=act)
    if c["op"] == "quantize":
        return _quantize_plain(s, c)
    if c["op"] == "linear":
        return _linear_plain(s, c)
    return _experts_plain(s, c)


def work(case):
    c = case
    T, K, block = c["T"], c["K"], BLOCK[c["format"]]
    value = 0.5 + 1.0 / block  # bytes
    if c["op"] == "quantize":  # there and back
        return dict(bytes=2 * T * K * (2 + value) + (8 if c["globals"] else 0), flops=4 * T * K)
    N = c["N"]
    out = N if c["act"] == "none" else N // 2
    if c["op"] == "linear":
        return dict(bytes=(N + T) * K * value + 4 + T * out * 2, flops=2 * T * N * K)
    n = T * c["k"]
    active = c["E"] * (1 - (1 - min(1.0, c["k"] / c["E"])) ** T)  # expected, with even experts
    return dict(bytes=active * N * K * value + (T if c["gather"] else n) * K * value + (n * 4 if c["gather"] else 0)
                + c["E"] * 12 + n * out * 2, flops=2 * n * N * K)


# ------------------------------------------------------------------ 64-bit definition


def _nearest(v, values, even):
    """Index of the value nearest to each v >= 0; between two, the one of `even`."""
    at = torch.bucketize(v, (values[1:] + values[:-1]) / 2)  # how many midpoints lie below v
    up = torch.zeros_like(v, dtype=torch.bool)
    middle = ((values[1:] + values[:-1]) / 2)[at.clamp(max=len(values) - 2)]
    up |= (v == middle) & (at < len(values) - 1) & ~even[at]
    return at + up


def _decoded(packed, byte, format):
    low, high = (packed & 15).long(), (packed >> 4).long()
    code = torch.stack([low, high], dim=-1).reshape(*packed.shape[:-1], -1)
    value = torch.tensor(MAGNITUDES, dtype=torch.float64, device=DEV)[code & 7] * (1 - 2 * (code >> 3))
    e, m = (byte >> 3).long(), (byte & 7).double()
    if format == "nvfp4":
        scale = torch.where(e > 0, torch.exp2(e.double() - 7) * (1 + m / 8), m / 512)
    else:
        scale = torch.exp2(byte.double() - 127)
    return value * scale.repeat_interleave(BLOCK[format], dim=-1)


def _silu_product(y, act):
    if act == "none":
        return y
    half = y.shape[-1] // 2
    gate, up = y[..., :half], y[..., half:]
    return gate * torch.special.expit(gate) * up


def exact(case, seed):
    global own
    c, was = case, own
    own = False  # the scales in their plain order
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if c["op"] == "quantize":
        x = s["x"].double()
        b = x.reshape(c["T"], -1, BLOCK[c["format"]])
        top = b.abs().max(dim=2).values
        even = torch.arange(127, device=DEV) % 2 == 0
        unit = 1.0 if s["g"] is None else float(s["g"].double())
        if c["format"] == "nvfp4":
            e4m3 = torch.tensor([m / 512 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8) for e in range(16) for m in range(8)][:127],
                                dtype=torch.float64, device=DEV)
            scale = e4m3[_nearest(top / unit / 6, e4m3, even)] * unit
        else:
            power = (top.float().view(torch.int32) >> 23) - 127  # floor(log2), from the bits (no logarithm to round)
            scale = torch.exp2(power.double() - 2).clamp(min=2.0 ** -127)
        grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=DEV)
        v = torch.where(scale[:, :, None] > 0, b.abs() / scale[:, :, None].clamp(min=1e-300), 0)
        return (grid[_nearest(v, grid, even[:8])] * torch.sign(b) * scale[:, :, None]).reshape(x.shape)
    x = _decoded(s["x"], s["x_scales"], c["format"])
    if c["op"] == "linear":
        y = torch.einsum("tk,nk->tn", x, _decoded(s["w"][0], s["w_scales"][0], c["format"]))
        return _silu_product(y * s["factor"].double(), c["act"])
    n, out = c["T"] * c["k"], c["N"] if c["act"] == "none" else c["N"] // 2
    y = torch.empty(n, out, dtype=torch.float64, device=DEV)
    ends = torch.cumsum(s["counts"], 0).tolist()
    for e in range(c["E"]):
        lo, hi = (ends[e - 1] if e else 0), ends[e]
        if hi > lo:
            rows = x[lo:hi] if s["row_token"] is None else x[s["row_token"][lo:hi].long()]
            w = _decoded(s["w"][e], s["w_scales"][e], c["format"])
            y[lo:hi] = _silu_product(torch.einsum("rk,nk->rn", rows, w) * s["factor"][e].double(), c["act"])
    return y
