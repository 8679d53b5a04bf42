"""The 4-bit microscaled (MXFP4) operators over the sizes they are used at.

Three operators, each in the call a user makes of the library (``own``) and in
a plain form of elementary torch operations in fp32:

* ``quantize``: a matrix to MXFP4 (E2M1 codes, two to a byte, and one E8M0
  scale per 32 elements of a row) and back to the values it stands for;
* ``linear``: y = x W^T with MXFP4 weights, the activations x quantized on
  entry to MXFP8 (E4M3 codes) or MXFP4, one scale per 32 elements of a row;
* ``layer``: the Mixture-of-Experts layer with MXFP4 expert weights and MXFP8
  activations: router logits, top-k, softmax of the chosen logits, SwiGLU
  experts, gate-weighted sum, and an always-on shared expert where there is one.

A block of 32 elements with the largest magnitude a has the scale 2^e,
e = max(floor(log2 a) - top, -127), top = 2 (E2M1) or 8 (E4M3), e = -127 for a
block of zeros; its elements are rounded to the nearest code value of v / 2^e,
ties to even, saturating at 6 (E2M1) or 448 (E4M3).
"""
import functools
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One token's row on its way into a 4-bit buffer: latency.
        dict(name="quantize_row", op="quantize", rows=1, cols=4096, dtype="bf16", gap=0),
        # Odd extents and a row stride of their own, fp32: a slice of a wider matrix.
        dict(name="quantize_odd", op="quantize", rows=1001, cols=1111, dtype="f32", gap=13),
        # Eight experts' gate matrices at load time: bandwidth.
        dict(name="quantize_experts", op="quantize", rows=8 * 1536, cols=4096, dtype="bf16", gap=0),
        # A projection of one decoded token: latency, then weight streaming.
        dict(name="linear_token", op="linear", T=1, N=4096, K=4096, act="mxfp8", gap=0),
        # A decode step's tokens through a wide projection: weight streaming.
        dict(name="linear_step", op="linear", T=48, N=16384, K=7168, act="mxfp8", gap=0),
        # Ragged in every extent, x a slice of a wider buffer.
        dict(name="linear_odd", op="linear", T=333, N=1000, K=1440, act="mxfp8", gap=24),
        # A prompt chunk through a square projection: tensor cores.
        dict(name="linear_chunk", op="linear", T=8192, N=4096, K=4096, act="mxfp8", gap=0),
        # The same with both operands in 4 bits.
        dict(name="linear_chunk4", op="linear", T=8192, N=4096, K=4096, act="mxfp4", gap=0),
        # A single decoded token through an expert layer: latency.
        dict(name="layer_token", op="layer", T=1, H=4096, E=128, k=8, I=1536, Is=0, zipf=0.0),
        # A decode step: streaming nearly every expert's weights.
        dict(name="layer_step", op="layer", T=64, H=4096, E=128, k=8, I=1536, Is=0, zipf=0.0),
        # Skewed loads: many experts with no token or a few, some with hundreds.
        dict(name="layer_skewed", op="layer", T=1024, H=4096, E=512, k=10, I=1024, Is=0, zipf=1.1),
        # A prompt chunk: tensor cores.
        dict(name="layer_chunk", op="layer", T=8192, H=4096, E=128, k=8, I=1536, Is=0, zipf=0.0),
    ]


def _log(rng, lo, hi, unit=1):
    """A size spread over the logarithm of [lo, hi] (in units), never 3072."""
    while True:
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        n = unit * max(lo, min(hi, n))
        if n != 3072:
            return n


def draw(rng):
    op = rng.choice(["quantize", "linear", "layer"])
    while True:
        if op == "quantize":
            c = dict(op=op, rows=_log(rng, 1, 20000), cols=_log(rng, 32, 16384),
                     dtype=rng.choice(["bf16", "f32"]), gap=rng.choice([0, 0, 1, 8, 40]))
            if c["rows"] * c["cols"] <= 50_000_000:
                return c
        elif op == "linear":
            c = dict(op=op, T=_log(rng, 1, 8192), N=_log(rng, 64, 16384), K=_log(rng, 64, 16384),
                     act=rng.choice(["mxfp8", "mxfp4"]), gap=rng.choice([0, 0, 1, 8, 40]))
            if c["T"] * c["N"] * c["K"] <= 8192 * 4096 * 4096 and c["N"] * c["K"] <= 2 ** 27:
                return c
        else:
            E = _log(rng, 4, 512)
            c = dict(op=op, T=_log(rng, 1, 8192), H=_log(rng, 2, 56, 128), E=E,
                     k=rng.randint(1, min(E, 10)), I=_log(rng, 1, 16, 128),
                     Is=rng.choice([0, 0, 128 * rng.randint(1, 16)]),
                     zipf=rng.choice([0.0, 0.0, 1.1]))
            if (c["H"] * E * c["I"] <= 128 * 4096 * 1536
                    and c["T"] * c["H"] * (c["k"] * c["I"] + c["Is"]) <= 8192 * 4096 * 8 * 1536):
                return c


# ---------------------------------------------------------------- inputs

def _activations(shape, gen):
    """Token rows with a few large channels, as hidden states have them."""
    x = torch.randn(shape, generator=gen, device=DEV)
    x[:, ::97] *= 6.0
    return x


def _weights(n, rows, cols, scale, gen):
    """MXFP4 matrices: codes [n * rows, 64 * ceil(cols / 128)] (two to a byte,
    the even element in the low half; zeros past the row's end) and scales, one
    byte per 32 elements in tiles of 128 rows x 4 blocks: 512 bytes, row r and
    block b at 16 * (r % 32) + 4 * (r // 32) + b, the tiles row-major."""
    kt = -(-cols // 128)
    q = torch.empty(n, rows, 64 * kt, dtype=torch.uint8, device=DEV)
    s = torch.empty(n, -(-rows // 128) * kt * 512, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (rows * cols))
    for a in range(0, n, step):
        w = torch.randn(min(step, n - a), rows, cols, generator=gen, device=DEV) * scale
        code, e = _encode4(w.to(torch.bfloat16).float())
        code = torch.nn.functional.pad(code, (0, 128 * kt - code.shape[-1]))
        q[a:a + step] = code[..., ::2] | (code[..., 1::2] << 4)
        b = torch.zeros(w.shape[0], -(-rows // 128) * 128, 4 * kt, dtype=torch.uint8, device=DEV)
        b[:, :rows, :e.shape[-1]] = (e + 127).to(torch.uint8)
        b = b.view(w.shape[0], -1, 4, 32, kt, 4).permute(0, 1, 4, 3, 2, 5)
        s[a:a + step] = b.reshape(w.shape[0], -1)
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "quantize":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        rows, cols = case["rows"], case["cols"]
        w = torch.randn(rows, cols + case["gap"], generator=gen, device=DEV)
        w *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=gen, device=DEV).float())
        return dict(case=case, src=w.to(dt)[:, :cols])
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        x = _activations((T, K + case["gap"]), gen).to(torch.bfloat16)[:, :K]
        q, s = _weights(1, N, K, 1 / math.sqrt(K), gen)
        st = dict(case=case, x=x, q=q[0], s=s[0])
        if own:
            import mixture_experts_layer_route_gb300 as moe
            st["linear"] = moe.LinearMXFP4.from_quantized(q[0], s[0], N, K, act=case["act"])
        return st
    T, H, E, k, I, Is = (case[n] for n in ("T", "H", "E", "k", "I", "Is"))
    wr = (torch.randn(E, H, generator=gen, device=DEV) / math.sqrt(H)).to(torch.bfloat16)
    bias = None
    if case["zipf"]:
        rank = torch.randperm(E, generator=gen, device=DEV).double() + 1
        bias = (-case["zipf"] * rank.log()).float()
    x = _activations((T, H), gen).to(torch.bfloat16)
    for _ in range(64):  # tokens whose choice of experts hangs on a rounding are drawn again
        lg = x.double() @ wr.double().t() + (0 if bias is None else bias.double())
        top = lg.topk(min(k + 1, E), dim=1).values
        bad = ((top[:, :-1] - top[:, 1:]) < 1e-3).any(1).nonzero().flatten()
        if bad.numel() == 0:
            break
        x[bad] = _activations((bad.numel(), H), gen).to(torch.bfloat16)
    # Gate and up rows alternate in runs of 64: [E][I / 64][gate, up][64][H].
    gu = _weights(E, 2 * I, H, 1 / math.sqrt(H), gen)
    dn = _weights(E, H, I, 1 / math.sqrt(I), gen)
    sgu = _weights(1, 2 * Is, H, 1 / math.sqrt(H), gen) if Is else None
    sdn = _weights(1, H, Is, 1 / math.sqrt(Is), gen) if Is else None
    st = dict(case=case, x=x, wr=wr, bias=bias, gu=gu, dn=dn, sgu=sgu, sdn=sdn)
    if own:
        import mixture_experts_layer_route_gb300 as moe
        st["layer"] = moe.MoELayerMXFP4.from_quantized(
            wr, gu, dn, k, router_bias=bias, shared_gate_up=sgu, shared_down=sdn)
    return st


# ---------------------------------------------------------------- plain forms

def _pow2(e):
    """2^e as fp32 from its bits, e in [-127, 127]."""
    e = e.to(torch.int32)
    return torch.where(e == -127, 1 << 22, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _blocks(v):
    """fp32 [..., cols] as blocks [..., nb, 32], zeros past the row's end."""
    v = torch.nn.functional.pad(v, (0, -v.shape[-1] % 32))
    return v.unflatten(-1, (-1, 32))


def _exponent(b, top):
    a = b.abs().amax(-1)
    return torch.where(a > 0, torch.frexp(a).exponent - 1 - top, -127).clamp(min=-127)


def _encode4(v):
    """E2M1 codes (uint8, [..., 32 nb]) and block exponents ([..., nb]) of fp32 rows."""
    b = _blocks(v)
    e = _exponent(b, 2)
    b = b * _pow2(-e)[..., None]
    a = b.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
         + (a >= 3.5) + (a > 5.0))
    return (c + 8 * (b < 0).to(torch.uint8)).flatten(-2), e


@functools.lru_cache(None)
def _table4(device):
    t = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(t + [-u for u in t], device=device)


def _values4(code):
    return _table4(code.device)[code.to(torch.int32)]


def _round4(v):
    code, e = _encode4(v)
    return (_blocks(_values4(code)) * _pow2(e)[..., None]).flatten(-2)[..., :v.shape[-1]]


def _round8(v):
    """fp32 rows to the values of their MXFP8 form."""
    b = _blocks(v)
    e = _exponent(b, 8)
    b = (b * _pow2(-e)[..., None]).clamp(-448.0, 448.0)
    step = _pow2(torch.where(b == 0, -9, (torch.frexp(b).exponent - 1).clamp(min=-6) - 3))
    return ((b / step).round() * step * _pow2(e)[..., None]).flatten(-2)[..., :v.shape[-1]]


def _expand(q, s, rows, cols):
    """fp32 [n, rows, cols] of MXFP4 matrices (codes [n, rows, ...], tiled scales)."""
    kt = q.shape[-1] // 64
    v = torch.stack([_values4(q & 15), _values4(q >> 4)], -1).flatten(-2)
    b = s.view(q.shape[0], -1, kt, 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
    b = b.reshape(q.shape[0], -1, 4 * kt)[:, :rows]
    v = v.view(q.shape[0], rows, 4 * kt, 32).mul_(_pow2(b.to(torch.int32) - 127)[..., None])
    return v.flatten(-2)[..., :cols]


def _plain_linear(st):
    c = st["case"]
    x = st["x"].float()
    x = _round8(x) if c["act"] == "mxfp8" else _round4(x)
    w = _expand(st["q"][None], st["s"][None], c["N"], c["K"])[0]
    return (x @ w.t()).to(torch.bfloat16)


def _silu_mul(g, u):
    return g / (1 + (-g).exp()) * u


def _experts(x, gu, dn, I, H):
    """Each of n experts on its own rows: x [n, m, H] (MXFP8 values) -> [n, m, H]."""
    w = _expand(*gu, 2 * I, H).unflatten(1, (-1, 2, 64))
    g = torch.bmm(x, w[:, :, 0].flatten(1, 2).transpose(1, 2))
    u = torch.bmm(x, w[:, :, 1].flatten(1, 2).transpose(1, 2))
    del w
    h = _round8(_silu_mul(g, u))
    return torch.bmm(h, _expand(*dn, H, I).transpose(1, 2))


def _plain_layer(st):
    c = st["case"]
    T, H, k, I, Is = (c[n] for n in ("T", "H", "k", "I", "Is"))
    x = st["x"].float()
    lg = x @ st["wr"].float().t()
    if st["bias"] is not None:
        lg = lg + st["bias"]
    top, ids = lg.sort(dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k].flatten()
    w = (top - top[:, :1]).exp()
    w = w / w.sum(1, keepdim=True)
    x = _round8(x)
    # Slots grouped by expert, every touched expert's rows padded to the longest.
    order = ids.argsort(stable=True)
    used, group, count = ids[order].unique_consecutive(return_inverse=True, return_counts=True)
    place = torch.arange(T * k, device=DEV) - (count.cumsum(0) - count)[group]
    xe = torch.zeros(used.numel(), int(count.max()), H, device=DEV)
    xe[group, place] = x[order // k]
    out = _experts(xe, [t[used] for t in st["gu"]], [t[used] for t in st["dn"]], I, H)
    y = torch.empty(T * k, H, device=DEV)
    y[order] = out[group, place]
    y = (y.view(T, k, H) * w[..., None]).sum(1)
    if Is:
        y = y + _experts(x[None], st["sgu"], st["sdn"], Is, H)[0]
    return y.to(torch.bfloat16)


def run(st):
    op = st["case"]["op"]
    if own:
        import mixture_experts_layer_route_gb300 as moe
        if op == "quantize":
            src = st["src"]
            q, s = moe.quantize_mxfp4_rows(src)
            return moe.dequantize_mxfp4_rows(q, s, src.shape[0], src.shape[1], dtype=src.dtype)
        return st["linear"](st["x"]) if op == "linear" else st["layer"](st["x"])
    if op == "quantize":
        return _round4(st["src"].float()).to(st["src"].dtype)
    return _plain_linear(st) if op == "linear" else _plain_layer(st)


# ---------------------------------------------------------------- bytes and operations

def work(case):
    c = case
    if c["op"] == "quantize":
        n, es = c["rows"] * c["cols"], 2 if c["dtype"] == "bf16" else 4
        # read, codes and scales written, the values written back
        return dict(bytes=n * (2 * es + 0.5 + 1 / 32), flops=0)
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        return dict(bytes=2 * T * K + N * K * (0.5 + 1 / 32) + 2 * T * N, flops=2 * T * N * K)
    T, H, E, k, I, Is = (c[n] for n in ("T", "H", "E", "k", "I", "Is"))
    p = [1.0] * E if not c["zipf"] else [(r + 1) ** -c["zipf"] for r in range(E)]
    total = sum(p)
    # experts that get a token, each token drawing k of them with these chances
    used = sum(1 - (1 - min(1.0, k * v / total)) ** T for v in p)
    weights = 3 * H * (used * I + Is) * (0.5 + 1 / 32) + 2 * E * H
    return dict(bytes=weights + 4 * T * H, flops=2 * T * H * (E + 3 * (k * I + Is)))


# ---------------------------------------------------------------- the definition in 64 bits

def _exact4(v):
    b = _blocks(v)
    a = b.abs().amax(-1, keepdim=True)
    p = torch.where(a > 0, torch.floor(torch.log2(a.clamp(min=1e-300))), -200.0)
    p = torch.where(torch.exp2(p + 1) <= a, p + 1, torch.where(torch.exp2(p) > a, p - 1, p))
    s = torch.exp2((p - 2).clamp(min=-127.0))
    m = (b / s).abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    r = ((m / step).round() * step).clamp(max=6.0) * s
    return torch.copysign(r, b).flatten(-2)[..., :v.shape[-1]]


def _exact8(v):
    b = _blocks(v)
    a = b.abs().amax(-1, keepdim=True)
    p = torch.where(a > 0, torch.floor(torch.log2(a.clamp(min=1e-300))), -200.0)
    p = torch.where(torch.exp2(p + 1) <= a, p + 1, torch.where(torch.exp2(p) > a, p - 1, p))
    s = torch.exp2((p - 8).clamp(min=-127.0))
    r = (b / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).double() * s
    return r.flatten(-2)[..., :v.shape[-1]]


def _exact_matrix(q, s, rows, cols):
    """float64 [rows, cols] of one MXFP4 matrix, from the layout's definition."""
    kt = -(-cols // 128)
    r = torch.arange(rows, device=DEV)[:, None]
    j = torch.arange(cols, device=DEV)[None, :]
    code = (q.view(rows, -1)[:, (j // 2)[0]] >> (4 * (j % 2)).to(torch.uint8)) & 15
    b = j // 32
    at = ((r // 128) * kt + b // 4) * 512 + 16 * (r % 32) + 4 * ((r % 128) // 32) + b % 4
    mag = (code & 7).double()
    mag = torch.where(mag < 2, mag * 0.5, torch.exp2((mag / 2).floor() - 1) * (1 + (mag % 2) / 2))
    mag = torch.where(code >= 8, -mag, mag)
    return mag * torch.exp2(s.view(-1)[at].double() - 127)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact4(st["src"].double())
    if case["op"] == "linear":
        x = st["x"].double()
        x = _exact8(x) if case["act"] == "mxfp8" else _exact4(x)
        return x @ _exact_matrix(st["q"], st["s"], case["N"], case["K"]).t()
    T, H, E, k, I, Is = (case[n] for n in ("T", "H", "E", "k", "I", "Is"))
    x = st["x"].double()
    lg = x @ st["wr"].double().t()
    if st["bias"] is not None:
        lg += st["bias"].double()
    top, ids = lg.topk(k, dim=1)
    w = torch.softmax(top, 1)
    x = _exact8(x)

    def expert(x, gu, dn, inner):
        m = _exact_matrix(*gu, 2 * inner, H).view(-1, 128, H)
        g, u = x @ m[:, :64].reshape(inner, H).t(), x @ m[:, 64:].reshape(inner, H).t()
        return _exact8(g * torch.sigmoid(g) * u) @ _exact_matrix(*dn, H, inner).t()

    y = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in range(E):
        t, r = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            part = expert(x[t], [v[e] for v in st["gu"]], [v[e] for v in st["dn"]], I)
            y[t] += part * w[t, r, None]
    if Is:
        y += expert(x, [v[0] for v in st["sgu"]], [v[0] for v in st["sdn"]], Is)
    return y
