"""The microscaled 4-bit linear layers and their gated feed-forward block, as cases to be measured.

Five operators belong together: the quantization of a matrix along its rows, its columns or both
from one read (``mq_mx4_quantize``, read back by ``mq_mx4_dequantize``), a linear layer on a
quantized weight (``mq_mx4_linear``) with both of its gradients (``mq_mx4_linear_backward``), and the
gated feed-forward product silu(x Wg^T) * (x Wu^T) (``mq_mx4_gated``) with its gradients
(``mq_mx4_gated_backward``).

A quantized matrix holds E2M1 codes with one power-of-two scale (a byte e, the value 2^(e - 127))
for each 32 elements of a row. Rows are cut into pieces of 256 columns: codes lie as
[piece][row][128] (two codes to a byte, the first in the low half), scales as [piece][row][8], the
columns past the last one filled with zeros.

``own`` false computes each operator in its plain form, elementary torch operations in 32 bits;
``own`` true makes the package's calls.
"""
import math

import torch

own = False

BLOCK = 32                 # elements that share a scale
PIECE = 256                # columns that lie together
E_MIN, E_MAX = 2, 252      # scale bytes: the smallest code step and the largest code are finite fp32 numbers
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # the activations of one generated token
        {"name": "quantize 1x4096 bf16 rows", "op": "quantize", "m": 1, "k": 4096,
         "dtype": "bf16", "rows": True, "cols": False},
        # an fp32 master weight, for the forward pass and for the gradient of its input
        {"name": "quantize 8192x4096 f32 both", "op": "quantize", "m": 8192, "k": 4096,
         "dtype": "f32", "rows": True, "cols": True},
        # a projection of one generated token: latency, then the weight's bytes
        {"name": "linear m1 k4096 n4096 bf16", "op": "linear", "m": 1, "k": 4096, "n": 4096,
         "dtype": "bf16", "out": "bf16"},
        # a small serving batch on a wide layer
        {"name": "linear m13 k8192 n5120 f16", "op": "linear", "m": 13, "k": 8192, "n": 5120,
         "dtype": "f16", "out": "f16"},
        # a chunk of a prompt of no even size, outputs kept in 32 bits
        {"name": "linear m333 k2000 n1111 bf16 f32", "op": "linear", "m": 333, "k": 2000,
         "n": 1111, "dtype": "bf16", "out": "f32"},
        # a batch of long prompts, or a training step's forward pass
        {"name": "linear m8192 k4096 n8192 bf16", "op": "linear", "m": 8192, "k": 4096, "n": 8192,
         "dtype": "bf16", "out": "bf16"},
        # gradients of a small layer on a short batch of no even size
        {"name": "linear_backward m500 k1536 n1000 f16", "op": "linear_backward", "m": 500,
         "k": 1536, "n": 1000, "dtype": "f16", "out": "f32"},
        # gradients of a square projection in a training step, the weight's in 32 bits
        {"name": "linear_backward m8192 k4096 n4096 bf16", "op": "linear_backward", "m": 8192,
         "k": 4096, "n": 4096, "dtype": "bf16", "out": "f32"},
        # the feed-forward block for a few generated tokens
        {"name": "gated m4 k4096 f11000 bf16", "op": "gated", "m": 4, "k": 4096, "n": 11000,
         "dtype": "bf16", "keep": False},
        # the feed-forward block of a training step, both projections kept for the backward pass
        {"name": "gated m4096 k4096 f8192 bf16 keep", "op": "gated", "m": 4096, "k": 4096,
         "n": 8192, "dtype": "bf16", "keep": True},
        # its gradients on a short batch
        {"name": "gated_backward m300 k1024 f2700 f16", "op": "gated_backward", "m": 300,
         "k": 1024, "n": 2700, "dtype": "f16"},
        # its gradients in a training step
        {"name": "gated_backward m4096 k4096 f8192 bf16", "op": "gated_backward", "m": 4096,
         "k": 4096, "n": 8192, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer's width: most are multiples of 64, some are not even."""
    w = _spread(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.6 else w


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "linear_backward", "gated", "gated_backward"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    m, k, n = _spread(rng, 1, 8192), _width(rng, 40, 8192), _width(rng, 40, 8192)
    if op == "quantize":
        rows = rng.random() < 0.7
        return {"op": op, "m": m, "k": min(k, 4096), "dtype": rng.choice(["bf16", "f16", "f32"]),
                "rows": rows, "cols": not rows or rng.random() < 0.6}
    if op == "linear":
        return {"op": op, "m": m, "k": min(k, 4096), "n": n,
                "dtype": rng.choice([dtype, dtype, "f32"]), "out": rng.choice([dtype, "f32"])}
    if op == "linear_backward":
        return {"op": op, "m": max(8, m), "k": min(k, 4096), "n": min(n, 4096), "dtype": dtype,
                "out": rng.choice([dtype, "f32"])}
    m, k = min(m, 4096), min(k, 4096)
    if op == "gated":
        return {"op": op, "m": m, "k": k, "n": n, "dtype": dtype, "keep": rng.random() < 0.4}
    return {"op": op, "m": max(8, m), "k": k, "n": n, "dtype": dtype}


# ---- inputs ----------------------------------------------------------------------------------

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _gen(seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    return g


def _activations(g, m, k, dtype):
    """Activations: rows of different sizes, a few columns far larger than the others."""
    x = torch.randn(m, k, generator=g, device=_device())
    x *= torch.exp(0.5 * torch.randn(m, 1, generator=g, device=_device()))
    x[:, ::97] *= 8.0
    return x.to(DTYPES[dtype])


def _gradients(g, m, n, dtype):
    """Gradients of a batch's mean loss: small, with heavy tails."""
    x = torch.randn(m, n, generator=g, device=_device())
    return (x * x.abs() * (2.0 ** -6)).to(DTYPES[dtype])


def _scale_bytes(amax):
    """Scale bytes of blocks with the largest magnitudes `amax` (fp32): the smallest power of two
    that brings them to 6 = 1.5 * 2^2 or less."""
    bits = amax.contiguous().view(torch.int32)
    e = (bits >> 23) - 2 + ((bits & 0x7FFFFF) > 0x400000).int()
    return torch.where((bits >> 23) == 255, torch.full_like(e, 255), e.clamp(E_MIN, E_MAX))


def _power(e):
    """2^e of whole numbers e, exact."""
    return torch.ldexp(torch.ones((), device=e.device), e)


def _grid(a):
    """Magnitudes a rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    step = 0.5 + 0.5 * (a >= 2).to(a.dtype) + (a >= 4).to(a.dtype)
    return (torch.round(a / step) * step).clamp(max=6.0)


def _blocks(x):
    """x [rows][columns] as [rows][blocks][32], the last block filled with zeros."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK)).view(x.shape[0], -1, BLOCK)


def _pack(x):
    """Codes and scale bytes of x [rows][columns] (fp32) as they are held."""
    rows, cols = x.shape
    pieces = -(-cols // PIECE)
    x = torch.nn.functional.pad(x, (0, pieces * PIECE - cols)).view(rows, -1, BLOCK)
    e = _scale_bytes(x.abs().amax(2))
    a = _grid(x.abs() * _power(127 - e)[..., None])
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4))
    code = (code.int() + 8 * torch.signbit(x).int()).view(rows, pieces, PIECE // 2, 2)
    codes = (code[..., 0] + 16 * code[..., 1]).to(torch.uint8)
    return {"codes": codes.transpose(0, 1).contiguous(),
            "scales": e.to(torch.uint8).view(rows, pieces, -1).transpose(0, 1).contiguous(),
            "cols": cols}


def _weight(g, rows, cols):
    """A weight [rows][columns] with rows of different sizes, in fp32."""
    w = torch.randn(rows, cols, generator=g, device=_device()) / math.sqrt(cols)
    return w * torch.exp(0.3 * torch.randn(rows, 1, generator=g, device=_device()))


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case, "op": op}
    m, k, n = case["m"], case["k"], case.get("n")
    new = lambda rows, cols, dtype: torch.empty(rows, cols, dtype=DTYPES[dtype], device=_device())
    if op == "quantize":
        s["x"] = _activations(g, m, k, case["dtype"])
        s["row"] = new(m, k, "bf16") if case["rows"] else None
        s["col"] = new(k, m, "bf16") if case["cols"] else None
        return s
    if op in ("linear", "gated"):
        s["x"] = _activations(g, m, k, case["dtype"])
        if op == "linear":
            s["w"] = _pack(_weight(g, n, k))
            s["y"] = new(m, n, case["out"])
            return s
        s["wg"], s["wu"] = _pack(_weight(g, n, k)), _pack(_weight(g, n, k))
        for name in ("h", "g", "u") if case["keep"] else ("h",):
            s[name] = new(m, n, case["dtype"])
        return s
    # what the forward pass left: the input's columns, the weights' columns
    s["x_col"] = _pack(_activations(g, m, k, "f32").t().contiguous())
    s["dx"] = new(m, k, case["dtype"])
    if op == "linear_backward":
        s["w_col"] = _pack(_weight(g, n, k).t().contiguous())
        s["dy"] = _gradients(g, m, n, case["dtype"])
        s["dw"] = new(n, k, case["out"])
        return s
    for name in ("wg", "wu"):
        s[name + "_col"] = _pack(_weight(g, n, k).t().contiguous())
        s["d" + name] = new(n, k, case["dtype"])
    s["dh"] = _gradients(g, m, n, case["dtype"])
    s["g"] = torch.randn(m, n, generator=g, device=_device()).mul_(1.5).to(DTYPES[case["dtype"]])
    s["u"] = torch.randn(m, n, generator=g, device=_device()).to(DTYPES[case["dtype"]])
    return s


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _handle(mq, s, name):
    """The package's handle of a quantized matrix, which a program makes once."""
    key = "handle " + name
    if key not in s:
        q = s[name]
        s[key] = mq.MX4(q["codes"].shape[1], q["cols"], q["codes"], q["scales"])
    return s[key]


def _own_quantize(s):
    import microscaling_quantized_convolution_amd as mq
    c = s["case"]
    if "q" not in s:
        s["q"] = (mq.MX4.empty(c["m"], c["k"], s["x"].device) if c["rows"] else None,
                  mq.MX4.empty(c["k"], c["m"], s["x"].device) if c["cols"] else None)
    row, col = s["q"]
    mq.mq_mx4_quantize(s["x"], row, col)
    out = {}
    if row is not None:
        out["row"] = mq.mq_mx4_dequantize(row, s["row"])
    if col is not None:
        out["col"] = mq.mq_mx4_dequantize(col, s["col"])
    return out


def _own_linear(s):
    import microscaling_quantized_convolution_amd as mq
    c = s["case"]
    if "ws" not in s:
        s["ws"] = mq.mx4_linear_workspace(c["m"], c["n"], c["k"], s["x"].device)
    mq.mq_mx4_linear(s["x"], _handle(mq, s, "w"), s["y"], s["ws"])
    return {"y": s["y"]}


def _own_linear_backward(s):
    import microscaling_quantized_convolution_amd as mq
    c = s["case"]
    if "ws" not in s:
        s["ws"] = mq.mx4_linear_backward_workspace(c["m"], c["n"], c["k"], s["dy"].device)
    mq.mq_mx4_linear_backward(s["dy"], _handle(mq, s, "x_col"), _handle(mq, s, "w_col"), s["dx"],
                              s["dw"], s["ws"])
    return {"dx": s["dx"], "dw": s["dw"]}


def _own_gated(s):
    import microscaling_quantized_convolution_amd as mq
    c = s["case"]
    if "ws" not in s:
        s["ws"] = mq.mx4_gated_workspace(c["m"], c["n"], c["k"], s["x"].device)
    mq.mq_mx4_gated(s["x"], _handle(mq, s, "wg"), _handle(mq, s, "wu"), s["h"], s["ws"],
                    s.get("g"), s.get("u"))
    return {name: s[name] for name in ("h", "g", "u") if name in s}


def _own_gated_backward(s):
    import microscaling_quantized_convolution_amd as mq
    c = s["case"]
    if "ws" not in s:
        s["ws"] = mq.mx4_gated_backward_workspace(c["m"], c["n"], c["k"], s["dh"].device)
    mq.mq_mx4_gated_backward(s["dh"], s["g"], s["u"], _handle(mq, s, "x_col"),
                             _handle(mq, s, "wg_col"), _handle(mq, s, "wu_col"), s["dx"],
                             s["dwg"], s["dwu"], s["ws"])
    return {"dx": s["dx"], "dwg": s["dwg"], "dwu": s["dwu"]}


# The plain forms. Held against exact(), which is written apart from them.

def _rounded(x):
    """The values that x [rows][columns] has once quantized along its rows, in fp32. (x in 64 bits
    is scaled and rounded there.)"""
    b = _blocks(x)
    e = _scale_bytes(b.abs().amax(2).float())
    p = _power(127 - e)[..., None]
    b = torch.copysign(_grid(b.abs() * p), b).float() * _power(e - 127)[..., None]
    return b.reshape(x.shape[0], -1)[:, :x.shape[1]]


def _pairs(device):
    """The two numbers that each byte of codes stands for."""
    v = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=device)
    v = torch.cat([v, -v])
    byte = torch.arange(256, device=device)
    return torch.stack([v[byte % 16], v[byte // 16]], 1)


def _values(q):
    """A quantized matrix in fp32."""
    pieces, rows, _ = q["codes"].shape
    v = _pairs(q["codes"].device)[q["codes"].int()].view(pieces, rows, PIECE // BLOCK, BLOCK)
    v *= _power(q["scales"].int() - 127)[..., None]
    return v.permute(1, 0, 2, 3).reshape(rows, pieces * PIECE)[:, :q["cols"]]


def _plain_quantize(s):
    x, out = s["x"].float(), {}
    if s["case"]["rows"]:
        out["row"] = _rounded(x).to(torch.bfloat16)
    if s["case"]["cols"]:
        out["col"] = _rounded(x.t().contiguous()).to(torch.bfloat16)
    return out


def _plain_linear(s):
    return {"y": (_rounded(s["x"].float()) @ _values(s["w"]).t()).to(s["y"].dtype)}


def _plain_linear_backward(s):
    dy = s["dy"].float()
    dx = _rounded(dy) @ _values(s["w_col"]).t()
    dw = _rounded(dy.t().contiguous()) @ _values(s["x_col"]).t()
    return {"dx": dx.to(s["dx"].dtype), "dw": dw.to(s["dw"].dtype)}


def _plain_gated(s):
    x = _rounded(s["x"].float())
    g, u = x @ _values(s["wg"]).t(), x @ _values(s["wu"]).t()
    out = {"h": g / (1 + torch.exp(-g)) * u, "g": g, "u": u}
    return {name: out[name].to(s[name].dtype) for name in out if name in s}


def _plain_gated_backward(s):
    # in 64 bits: a value next to the border of two codes falls to either of them
    g, u, dh = s["g"].double(), s["u"].double(), s["dh"].double()
    sig = 1 / (1 + torch.exp(-g))
    dg, du = dh * u * sig * (1 + g * (1 - sig)), dh * g * sig
    dx = _rounded(dg) @ _values(s["wg_col"]).t() + _rounded(du) @ _values(s["wu_col"]).t()
    x = _values(s["x_col"]).t()
    dwg, dwu = _rounded(dg.t().contiguous()) @ x, _rounded(du.t().contiguous()) @ x
    return {"dx": dx.to(s["dx"].dtype), "dwg": dwg.to(s["dwg"].dtype), "dwu": dwu.to(s["dwu"].dtype)}


_plain = {"quantize": _plain_quantize, "linear": _plain_linear,
          "linear_backward": _plain_linear_backward, "gated": _plain_gated,
          "gated_backward": _plain_gated_backward}
_own = {"quantize": _own_quantize, "linear": _own_linear,
        "linear_backward": _own_linear_backward, "gated": _own_gated,
        "gated_backward": _own_gated_backward}


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    op, m, k, n = case["op"], case["m"], case["k"], case.get("n", 0)
    held, size = 17.0 / 32, SIZES[case["dtype"]]   # bytes of a quantized element, of another one
    if op == "quantize":  # written, and read back as bf16
        ways = case["rows"] + case["cols"]
        return {"bytes": m * k * (size + ways * (2 * held + 2)), "flops": 4 * ways * m * k}
    if op == "linear":
        return {"bytes": m * k * size + n * k * held + m * n * SIZES[case["out"]],
                "flops": 2 * m * n * k}
    if op == "linear_backward":
        return {"bytes": m * n * size + (m + n) * k * held + m * k * size
                + n * k * SIZES[case["out"]], "flops": 4 * m * n * k}
    if op == "gated":
        return {"bytes": m * k * size + 2 * n * k * held + m * n * size * (3 if case["keep"] else 1),
                "flops": 4 * m * n * k}
    return {"bytes": 3 * m * n * size + (m + 2 * n) * k * held + (m + 2 * n) * k * size,
            "flops": 8 * m * n * k}


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _exact_quantize, "linear": _exact_linear,
            "linear_backward": _exact_linear_backward, "gated": _exact_gated,
            "gated_backward": _exact_gated_backward}[case["op"]](s)


def _exact_rounded(x):
    """Each 32 of a row (64 bits) to the nearest element of the grid at their scale."""
    rows, cols = x.shape
    out = torch.zeros(rows, -(-cols // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    out[:, :cols] = x
    out = out.view(rows, -1, BLOCK)
    top = out.abs().max(2, keepdim=True).values
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 6)).clamp(E_MIN - 127, E_MAX - 127))
    # log2 rounds: put right what it left a step too small or too large
    scale = torch.where(top > 6 * scale, 2 * scale, scale)
    scale = torch.where((top <= 3 * scale) & (scale > 2.0 ** (E_MIN - 127)), scale / 2, scale)
    a, sign = (out / scale).abs(), torch.sign(out)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    # between two elements: up past the middle, at the middle to the even one
    edge = (grid[1:] + grid[:-1]) / 2
    up, down = torch.bucketize(a, edge, right=True), torch.bucketize(a, edge)
    code = torch.where(up % 2 == 0, up, down)
    return (sign * grid[code] * scale).reshape(rows, -1)[:, :cols]


def _exact_values(q):
    """A quantized matrix in 64 bits, from the bits of its codes: sign, two of exponent, one of
    fraction."""
    pieces, rows, _ = q["codes"].shape
    out = torch.empty(rows, pieces * PIECE, dtype=torch.float64, device=q["codes"].device)
    for p in range(pieces):
        for half in (0, 1):
            c = (q["codes"][p] >> (4 * half)) & 15
            power, frac = ((c >> 1) & 3).double(), (c & 1).double()
            v = torch.where(power > 0, (1 + frac / 2) * torch.exp2(power - 1), frac / 2)
            v = torch.where(c >= 8, -v, v)
            e = q["scales"][p].double().repeat_interleave(BLOCK // 2, 1)
            out[:, p * PIECE + half:(p + 1) * PIECE:2] = v * torch.exp2(e - 127)
    return out[:, :q["cols"]]


def _exact_quantize(s):
    x, c = s["x"].double(), s["case"]
    out = {"row": _exact_rounded(x)} if c["rows"] else {}
    if c["cols"]:
        out["col"] = _exact_rounded(x.t())
    return out


def _exact_linear(s):
    return {"y": torch.mm(_exact_rounded(s["x"].double()), _exact_values(s["w"]).t().contiguous())}


def _exact_linear_backward(s):
    dy = s["dy"].double()
    return {"dx": torch.mm(_exact_rounded(dy), _exact_values(s["w_col"]).t().contiguous()),
            "dw": torch.mm(_exact_rounded(dy.t()), _exact_values(s["x_col"]).t().contiguous())}


def _exact_gated(s):
    x = _exact_rounded(s["x"].double())
    g = torch.mm(x, _exact_values(s["wg"]).t().contiguous())
    u = torch.mm(x, _exact_values(s["wu"]).t().contiguous())
    out = {"h": g * torch.sigmoid(g) * u, "g": g, "u": u}
    return {name: out[name] for name in out if name in s}


def _exact_gated_backward(s):
    g, u, dh = s["g"].double(), s["u"].double(), s["dh"].double()
    sig = torch.sigmoid(g)
    d = {"wg": dh * u * (sig + g * sig * (1 - sig)), "wu": dh * g * sig}
    x, out = _exact_values(s["x_col"]).t().contiguous(), {}
    out["dx"] = sum(torch.mm(_exact_rounded(d[w]), _exact_values(s[w + "_col"]).t().contiguous())
                    for w in d)
    for w in d:
        out["d" + w] = torch.mm(_exact_rounded(d[w].t()), x)
    return out
