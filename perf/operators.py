"""The 8-bit operators of a rotated layer, as cases that can be measured.

A rotated layer keeps its activations and weights as E4M3 codes with one scale
for each block of 128: rows are quantised in blocks of 1 x 128, weights in
blocks of 128 x 128.  Scales are fp32 or powers of two (E8M0).  A block's scale
is its largest magnitude over 448 (E8M0: rounded up to a power of two), never
below 2^-120, and its codes are the values over the scale, rounded to nearest
even.

  quantise   codes and scales of rows (a checkpoint) or of a weight
  norm       h = x + residual, then the root-mean-square norm of h, as codes;
             with checkpoint, also 1/rms and the codes of h/rms
  norm_grad  dh and dgamma of the norm, from the checkpoint's codes
  matmul     y = A W^T of two coded matrices
  wgrad      dW = dY^T X with X from the checkpoint's codes

`own` chooses between the plain form (torch, fp32) and the library's calls.
"""
import math

import torch

own = False

BLK = 128
TOP = 448.0                 # largest E4M3 value
FLOOR = 2.0 ** -120         # smallest scale
EPS = 1e-6
_SDT = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}
_IO = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a calibration batch of rotated activations kept as a checkpoint
        {"name": "quantise rows 16384x4096", "op": "quantise", "rows": 16384, "cols": 4096, "tile": 1,
         "scale": "f32", "io": "bf16"},
        # a rotated weight stored once, before serving
        {"name": "quantise weight 13824x5120", "op": "quantise", "rows": 13824, "cols": 5120, "tile": 128,
         "scale": "e8m0", "io": "bf16"},
        # one token of decoding, rotated stream (the norm's weight folded into W): latency
        {"name": "norm 1x4096", "op": "norm", "rows": 1, "cols": 4096, "scale": "f32", "io": "bf16",
         "gamma": False, "checkpoint": False},
        # a calibration batch: the norm's own weight, and the checkpoint for the backward pass
        {"name": "norm 16384x5120 checkpoint", "op": "norm", "rows": 16384, "cols": 5120, "scale": "e8m0",
         "io": "bf16", "gamma": True, "checkpoint": True},
        # the same batch's backward pass
        {"name": "norm_grad 16384x5120", "op": "norm_grad", "rows": 16384, "cols": 5120, "scale": "e8m0",
         "io": "bf16", "gamma": True},
        # a ragged batch of fp32 rows, odd length, a rotated stream
        {"name": "norm_grad 1021x4099 f32", "op": "norm_grad", "rows": 1021, "cols": 4099, "scale": "f32",
         "io": "f32", "gamma": False},
        # one token of decoding through a square layer: latency, and the weight's bytes
        {"name": "matmul 1x4096x4096", "op": "matmul", "rows": 1, "n": 4096, "k": 4096, "scale": "f32",
         "out": "bf16"},
        # a batch of decoding requests through the widest layer
        {"name": "matmul 64x13824x5120", "op": "matmul", "rows": 64, "n": 13824, "k": 5120, "scale": "e8m0",
         "out": "bf16"},
        # a ragged prompt; the reduction ends inside a block
        {"name": "matmul 777x5120x4112 f32", "op": "matmul", "rows": 777, "n": 5120, "k": 4112, "scale": "f32",
         "out": "f32"},
        # a calibration batch through the widest layer, fp32 scales
        {"name": "matmul 16384x13824x5120", "op": "matmul", "rows": 16384, "n": 13824, "k": 5120,
         "scale": "f32", "out": "bf16"},
        # the weight's gradient of a calibration batch, powers of two as scales, fp32 result
        {"name": "wgrad 16384x4096x4096", "op": "wgrad", "rows": 16384, "n": 4096, "k": 4096, "scale": "e8m0",
         "out": "f32"},
        # a ragged batch into odd sizes, fp32 scales, bf16 result
        {"name": "wgrad 1500x4099x1037", "op": "wgrad", "rows": 1500, "n": 4099, "k": 1037, "scale": "f32",
         "out": "bf16"},
    ]


def _spread(rng, lo, hi, step=1):
    """A size spread over the logarithm of lo..hi, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    v = min(max(v, lo), hi)
    return v + step if v == 3 * 1024 else v


def draw(rng):
    op = rng.choice(["quantise", "norm", "norm_grad", "matmul", "matmul", "wgrad"])
    c = {"op": op, "scale": rng.choice(["f32", "e8m0"])}
    if op in ("matmul", "wgrad"):
        # rows of 16-byte pieces (every size of a model) three times in four, else any length
        step = 16 if rng.random() < 0.75 else 1
        c["rows"] = _spread(rng, 1, 16384)
        c["n"] = _spread(rng, 64, 13824, step)
        c["k"] = _spread(rng, 64, 5120, step)
        c["out"] = rng.choice(["bf16", "f32"])
        return c
    c["rows"] = _spread(rng, 1, 16384)
    c["cols"] = _spread(rng, 64, 8192, 8 if rng.random() < 0.75 else 1)
    c["io"] = rng.choice(["bf16", "f32"])
    if op == "quantise":
        c["tile"] = rng.choice([1, 128])
    else:
        c["gamma"] = rng.random() < 0.5
    if op == "norm":
        c["checkpoint"] = rng.random() < 0.5
    return c


# ----------------------------------------------------------------- inputs
def _nblk(n):
    return (n + BLK - 1) // BLK


def _heavy(g, rows, cols, channels=0):
    """Student-t rows (3 degrees of freedom), some channels 50 times larger."""
    z = torch.randn(rows, cols, generator=g, device="cuda")
    chi = torch.zeros(rows, cols, device="cuda")
    for _ in range(3):
        chi += torch.randn(rows, cols, generator=g, device="cuda") ** 2
    z *= torch.sqrt(3.0 / chi.clamp_(min=1e-6))
    if channels:
        at = torch.randperm(cols, generator=g, device="cuda")[:channels]
        z[:, at] *= 50.0
    return z


def _coded(x, tile, scale):
    """Codes and scales of x, made for an operator that takes them as inputs."""
    return _plain_quantise(x, tile, scale)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, rows = case["op"], case["rows"]
    s = dict(case)
    if op == "quantise":
        io = _IO[case["io"]]
        if case["tile"] == 1:
            s["x"] = _heavy(g, rows, case["cols"], case["cols"] // 100).to(io)
            s["x"][rows - rows // 64:] = 0            # padding of the batch
        else:
            s["x"] = (torch.randn(rows, case["cols"], generator=g, device="cuda") * 0.02).to(io)
    elif op == "norm":
        io = _IO[case["io"]]
        s["x"] = _heavy(g, rows, case["cols"]).to(io)
        s["residual"] = _heavy(g, rows, case["cols"], case["cols"] // 100).to(io)
        s["weight"] = (1.0 + 0.2 * torch.randn(case["cols"], generator=g, device="cuda")).to(io) if case["gamma"] \
            else None
    elif op == "norm_grad":
        io = _IO[case["io"]]
        h = _heavy(g, rows, case["cols"], case["cols"] // 100)
        r = torch.rsqrt((h * h).mean(1) + EPS)
        s["codes"], s["scales"] = _coded(h * r[:, None], 1, case["scale"])
        s["rstd"] = r
        s["dn"] = (_heavy(g, rows, case["cols"]) * 1e-3).to(io)
        s["dres"] = (_heavy(g, rows, case["cols"]) * 1e-3).to(io)
        s["weight"] = (1.0 + 0.2 * torch.randn(case["cols"], generator=g, device="cuda")).to(io) if case["gamma"] \
            else None
    elif op == "matmul":
        # rotated activations and weights: close to normal, whatever they were before
        a = torch.randn(rows, case["k"], generator=g, device="cuda")
        a *= torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))
        s["a"], s["a_scales"] = _coded(a, 1, case["scale"])
        w = torch.randn(case["n"], case["k"], generator=g, device="cuda") * 0.02
        s["w"], s["w_scales"] = _coded(w, BLK, case["scale"])
    else:
        x = torch.randn(rows, case["k"], generator=g, device="cuda")
        s["x"], s["x_scales"] = _coded(x, 1, case["scale"])
        s["dy"] = (_heavy(g, rows, case["n"]) * 1e-3).to(torch.bfloat16)
    _buffers(s)
    return s


def _buffers(s):
    """The output buffers that a program keeps from call to call."""
    rows = s["rows"]
    if s["op"] == "quantise":
        s["codes"] = torch.empty(rows, s["cols"], dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty(-(-rows // s["tile"]), _nblk(s["cols"]), dtype=_SDT[s["scale"]], device="cuda")
    elif s["op"] == "norm":
        s["codes"] = torch.empty(rows, s["cols"], dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty(rows, _nblk(s["cols"]), dtype=_SDT[s["scale"]], device="cuda")
        s["h"] = torch.empty_like(s["x"])
    elif s["op"] == "norm_grad":
        s["dh"] = torch.empty_like(s["dn"])
    elif s["op"] == "matmul":
        s["y"] = torch.empty(rows, s["n"], dtype=_IO[s["out"]], device="cuda")
    else:
        s["dw"] = torch.empty(s["n"], s["k"], dtype=_IO[s["out"]], device="cuda")


# -------------------------------------------------------------- one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import structured_rotations_amd as lib
    op = s["op"]
    if op == "quantise":
        return lib.harp_quantize_q8(s["x"], s["tile"], s["scale"], codes=s["codes"], scales=s["scales"])
    if op == "norm":
        r = lib.harp_rmsnorm_q8(s["x"], s["residual"], s["weight"], EPS, s["scale"], checkpoint=s["checkpoint"],
                                h=s["h"], codes=s["codes"], scales=s["scales"])
        out = {"codes": r.codes, "scales": r.scales, "h": r.h}
        if s["checkpoint"]:
            out |= {"rstd": r.rstd, "ckpt_codes": r.ckpt_codes, "ckpt_scales": r.ckpt_scales}
        return out
    if op == "norm_grad":
        return lib.harp_rmsnorm_q8_vjp(s["codes"], s["scales"], s["rstd"], s["dn"], s["weight"], s["dres"],
                                       dh=s["dh"])
    if op == "matmul":
        return lib.harp_matmul_q8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["out"], y=s["y"])
    return lib.harp_matmul_q8_wgrad(s["dy"], s["x"], s["x_scales"], s["out"], dw=s["dw"])


def _plain(s):
    op = s["op"]
    if op == "quantise":
        return _plain_quantise(s["x"].float(), s["tile"], s["scale"])
    if op == "norm":
        h = s["x"].float() + s["residual"].float()
        r = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
        xn = h * r[:, None]
        n = xn if s["weight"] is None else xn * s["weight"].float()
        codes, scales = _plain_quantise(n, 1, s["scale"])
        out = {"codes": codes, "scales": scales, "h": h.to(s["x"].dtype)}
        if s["checkpoint"]:
            ck = (codes, scales) if s["weight"] is None else _plain_quantise(xn, 1, s["scale"])
            out |= {"rstd": r, "ckpt_codes": ck[0], "ckpt_scales": ck[1]}
        return out
    if op == "norm_grad":
        xn = _plain_values(s["codes"], s["scales"], 1)
        dn = s["dn"].float()
        gdn = dn if s["weight"] is None else dn * s["weight"].float()
        dh = s["dres"].float() + s["rstd"][:, None] * (gdn - xn * (gdn * xn).mean(1, keepdim=True))
        dgamma = None if s["weight"] is None else (dn * xn).sum(0)
        return dh.to(s["dn"].dtype), dgamma
    if op == "matmul":
        a = _plain_values(s["a"], s["a_scales"], 1)
        w = _plain_values(s["w"], s["w_scales"], BLK)
        return torch.matmul(a, w.t()).to(_IO[s["out"]])
    x = _plain_values(s["x"], s["x_scales"], 1)
    return torch.matmul(s["dy"].float().t(), x).to(_IO[s["out"]])


def _plain_quantise(x, tile, scale):
    rows, cols = x.shape
    nr, nc = -(-rows // tile), _nblk(cols)
    p = torch.nn.functional.pad(x.float(), (0, nc * BLK - cols, 0, nr * tile - rows)).view(nr, tile, nc, BLK)
    s = (p.abs().amax(dim=(1, 3)) / TOP).clamp(min=FLOOR)
    if scale == "e8m0":
        m, e = torch.frexp(s)                                   # s = m 2^e, 1/2 <= m < 1
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    codes = (p * (1.0 / s)[:, None, :, None]).view(nr * tile, nc * BLK)[:rows, :cols].to(torch.float8_e4m3fn)
    return codes, s.to(_SDT[scale])


def _plain_values(codes, scales, tile):
    rows, cols = codes.shape
    s = scales.float()
    s = s if tile == 1 else s.repeat_interleave(tile, 0)[:rows]
    return codes.float() * s.repeat_interleave(BLK, 1)[:, :cols]


# ------------------------------------------------------------------- work
def work(case):
    rows = case["rows"]
    sb = 4 if case["scale"] == "f32" else 1
    if case["op"] == "quantise":
        n, eb = rows * case["cols"], 4 if case["io"] == "f32" else 2
        return {"bytes": n * (eb + 1) + sb * -(-rows // case["tile"]) * _nblk(case["cols"]), "flops": 2 * n}
    if case["op"] == "norm":
        n, eb = rows * case["cols"], 4 if case["io"] == "f32" else 2
        b = n * (3 * eb + 1) + sb * rows * _nblk(case["cols"]) + eb * case["cols"] * case["gamma"]
        if case["checkpoint"]:
            b += 4 * rows + case["gamma"] * (n + sb * rows * _nblk(case["cols"]))
        return {"bytes": b, "flops": 6 * n}
    if case["op"] == "norm_grad":
        n, eb = rows * case["cols"], 4 if case["io"] == "f32" else 2
        b = n * (3 * eb + 1) + sb * rows * _nblk(case["cols"]) + 4 * rows
        return {"bytes": b + (eb + 4) * case["cols"] * case["gamma"], "flops": 8 * n}
    n, k = case["n"], case["k"]
    ob = 4 if case["out"] == "f32" else 2
    if case["op"] == "matmul":
        b = rows * k + n * k + sb * (rows + _nblk(n)) * _nblk(k) + ob * rows * n
    else:
        b = rows * k + 2 * rows * n + sb * rows * _nblk(k) + ob * n * k
    return {"bytes": b, "flops": 2 * rows * n * k}


# ------------------------------------------------- the definition, 64 bits
def _values64(codes, scales, tile):
    """sum over blocks of 128 columns, each block's codes times its scale."""
    v = codes.to(torch.float64)
    s = scales.to(torch.float64)
    for j in range(s.shape[1]):
        col = s[:, j] if tile == 1 else s[torch.arange(v.shape[0], device=v.device) // tile, j]
        v[:, j * BLK:(j + 1) * BLK] *= col[:, None]
    return v


def _quantise64(x, tile, scale):
    rows, cols = x.shape
    codes = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=x.device)
    out = torch.empty(-(-rows // tile), _nblk(cols), dtype=torch.float64, device=x.device)
    for j in range(_nblk(cols)):
        b = x[:, j * BLK:(j + 1) * BLK]
        top = torch.zeros(out.shape[0], dtype=torch.float64, device=x.device)
        top.scatter_reduce_(0, torch.arange(rows, device=x.device) // tile, b.abs().max(1).values, "amax")
        s = torch.clamp(top / 448.0, min=2.0 ** -120)
        if scale == "e8m0":
            s = torch.exp2(torch.ceil(torch.log2(s)))
        out[:, j] = s
        v = b / s[torch.arange(rows, device=x.device) // tile][:, None]
        # E4M3 values: 4 significant bits down to 2^-6, steps of 2^-9 below; round to even
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs().clamp(min=1e-30))), min=-6.0) - 3.0)
        codes[:, j * BLK:(j + 1) * BLK] = (torch.round(v / step) * step).float().to(torch.float8_e4m3fn)
    return codes, out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        return _quantise64(s["x"].double(), case["tile"], case["scale"])
    if op == "norm":
        h = s["x"].double() + s["residual"].double()
        r = (h.square().sum(1) / case["cols"] + EPS) ** -0.5
        xn = h * r[:, None]
        codes, scales = _quantise64(xn * s["weight"].double() if case["gamma"] else xn, 1, case["scale"])
        out = {"codes": codes, "scales": scales, "h": h}
        if case["checkpoint"]:
            ck = _quantise64(xn, 1, case["scale"])
            out |= {"rstd": r, "ckpt_codes": ck[0], "ckpt_scales": ck[1]}
        return out
    if op == "norm_grad":
        xn = _values64(s["codes"], s["scales"], 1)
        up = s["dn"].double()
        dgamma = (up * xn).sum(0) if case["gamma"] else None
        if case["gamma"]:
            up = up * s["weight"].double()
        r = s["rstd"].double()[:, None]
        along = (up * xn).sum(1, keepdim=True) / case["cols"]
        return s["dres"].double() + up * r - xn * along * r, dgamma
    if op == "matmul":
        w = _values64(s["w"], s["w_scales"], BLK)
        return torch.mm(_values64(s["a"], s["a_scales"], 1), w.T.contiguous())
    return torch.mm(s["dy"].double().T.contiguous(), _values64(s["x"], s["x_scales"], 1))
