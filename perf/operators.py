"""What the fused-epilogue and 8-bit-checkpoint operators of libqlora cost.

One layer is y = act(x deq(W) + s (x A) B + bias) + residual with a frozen
quantized W [K, N] and a float32 adapter A [K, r], B [r, N], s = alpha / r.
The operators:

* ``fwd``     the product with its epilogue; the pre-activation z and the
              8-bit row checkpoint of x are saved on the way where asked for;
* ``refwd``   the same output again from the row checkpoint of x (the second
              forward of a checkpointed block);
* ``bwd``     dx, dA and dB with x as its 8-bit row checkpoint; dx may be
              carried through the activation that made x (act'(z), z as an
              8-bit group checkpoint) and the skip connection's gradient
              added;
* ``actbwd``  dz = dy act'(z) and the bias gradient, on their own;
* ``ckpt``    an activation written to 8 bits and read back.

8-bit forms. Rows ("c8row"): codes round-half-even(x * (127 / absmax)), one
float32 scale absmax / 127 per row, in float32 operations. Groups ("c8g32"):
32 consecutive columns share a power of two 2^e, the smallest with
absmax <= 127 2^e (kept as the byte e + 127), codes round-half-even(v 2^-e)
but at least 1 in size where v is not 0, so that a sign is never lost (the
slope of a ReLU is then that of the value before it was written).
"""

import math

import torch

own = False

GROUP = 32                      # columns per scale of a group checkpoint
W4_GROUP = 128                  # inputs per scale of a 4-bit weight


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a small float32 layer with a ReLU: all latency
        dict(name="fwd f32 64x256x256 relu", op="fwd", fmt="w8", dtype="f32", M=64, K=256, N=256, r=4,
             act="relu", bias=True, residual=False, save_x=False, save_z="full"),
        # one token through a wide decoder feed-forward (serving)
        dict(name="fwd 1x2048x16384 gelu", op="fwd", fmt="w8", dtype="bf16", M=1, K=2048, N=16384, r=8,
             act="gelu_tanh", bias=True, residual=False, save_x=False, save_z="none"),
        # a GPT-2-sized projection at 32 sequences of 128 tokens, everything
        # that its backward needs saved in 8 bits
        dict(name="fwd 4096x768x2304 gelu c8", op="fwd", fmt="w8", dtype="bf16", M=4096, K=768, N=2304, r=4,
             act="gelu", bias=True, residual=False, save_x=True, save_z="c8g32"),
        # the 4-bit 4096 x 4096 layer inside a residual block
        dict(name="fwd w4 2048x4096x4096 silu+res", op="fwd", fmt="w4g128", dtype="bf16", M=2048, K=4096, N=4096, r=4,
             act="silu", bias=False, residual=True, save_x=False, save_z="full"),
        # a ragged last batch of the 1024-wide MLP: odd rows, skip connection
        dict(name="fwd 1001x784x1024 relu+res", op="fwd", fmt="w8", dtype="bf16", M=1001, K=784, N=1024, r=8,
             act="relu", bias=True, residual=True, save_x=True, save_z="none"),
        # second forward of a checkpointed decoder block: the down projection
        dict(name="refwd 512x16384x2048 res", op="refwd", fmt="w8", dtype="bf16", M=512, K=16384, N=2048, r=8,
             act="none", bias=True, residual=True, save_x=False, save_z="none"),
        # one layer of the 1024-wide MLP, backward through its ReLU
        dict(name="bwd 1024x1024x1024 relu", op="bwd", fmt="w8", dtype="bf16", M=1024, K=1024, N=1024, r=8,
             act="relu", add=False),
        # a GPT-2-sized projection whose input also feeds the skip connection
        dict(name="bwd 4096x768x2304 add", op="bwd", fmt="w8", dtype="bf16", M=4096, K=768, N=2304, r=4,
             act="none", add=True),
        # the down projection of the decoder feed-forward, through its GELU
        dict(name="bwd 512x16384x2048 gelu", op="bwd", fmt="w8", dtype="bf16", M=512, K=16384, N=2048, r=8,
             act="gelu_tanh", add=False),
        # activation and bias gradient of a layer whose consumer is not one of these
        dict(name="actbwd 4096x2304 gelu", op="actbwd", dtype="bf16", M=4096, C=2304, act="gelu"),
        dict(name="actbwd f32 77x1040 silu", op="actbwd", dtype="f32", M=77, C=1040, act="silu"),
        # the cached input of a decoder block: 512 tokens, its feed-forward width
        dict(name="ckpt g32 512x16384", op="ckpt", cfmt="c8g32", dtype="bf16", M=512, C=16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
MOST_MACS = 2048 * 4096 * 4096          # the largest listed product


def draw(rng):
    op = rng.choice(["fwd", "fwd", "refwd", "bwd", "bwd", "actbwd", "ckpt"])
    f32 = rng.random() < 0.2
    M = _log(rng, 1, 4096)
    if op in ("actbwd", "ckpt"):
        C = 16 * _log(rng, 1, 1024)
        M = min(M, 16 * 1024 * 1024 // C)
        c = dict(op=op, dtype="f32" if f32 else "bf16", M=M, C=C)
        c.update(act=rng.choice(ACTS[1:])) if op == "actbwd" else c.update(cfmt=rng.choice(["c8row", "c8g32"]))
        return c
    fmt = "w8" if f32 else rng.choice(["w8", "w8", "w4g128"])
    unit = 128 if fmt == "w4g128" else 16
    top = 512 if f32 else 16384
    K = unit * _log(rng, 1, top // unit)
    N = 16 * _log(rng, 1, top // 16)
    M = max(1, min(M, MOST_MACS // (K * N), 16 * 1024 * 1024 // max(K, N), 512 if f32 else M))
    c = dict(op=op, fmt=fmt, dtype="f32" if f32 else "bf16", M=M, K=K, N=N, r=rng.choice([1, 3, 4, 8, 8, 16, 32]),
             act=rng.choice(ACTS))
    if op == "bwd":
        c.update(add=rng.random() < 0.5)
    else:
        c.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5, save_x=op == "fwd" and rng.random() < 0.5,
                 save_z=rng.choice(["none", "full", "c8g32"]))
    return c


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    M = case["M"]
    c8 = 1 + 1 / GROUP
    if case["op"] == "actbwd":
        C = case["C"]
        return dict(bytes=M * C * (2 * e + c8) + 4 * C, flops=20 * M * C)
    if case["op"] == "ckpt":
        return dict(bytes=M * case["C"] * (2 * e + 2 * c8), flops=4 * M * case["C"])
    K, N, r = case["K"], case["N"], case["r"]
    weight = K * N + 4 * N if case["fmt"] == "w8" else K * N // 2 + 2 * N * (K // W4_GROUP)
    adapter = 4 * r * (K + N)
    if case["op"] == "bwd":
        b = weight + 2 * adapter + 4 * M * r + M * (K + 4) + e * M * (N + K)
        b += (M * K * c8 if case["act"] != "none" else 0) + (e * M * K if case["add"] else 0)
        return dict(bytes=b, flops=2 * M * K * N + 8 * M * r * (K + N))
    x8 = M * (K + 4)
    b = weight + adapter + 4 * M * r + (x8 if case["op"] == "refwd" else e * M * K) + e * M * N
    b += 4 * N if case["bias"] else 0
    b += e * M * N if case["residual"] else 0
    b += x8 if case["save_x"] else 0
    b += {"none": 0, "full": e * M * N, "c8g32": M * N * c8}[case["save_z"]]
    return dict(bytes=b, flops=2 * M * K * N + 2 * M * r * (K + N))


# ---------------------------------------------------------------------------
# the 8-bit forms in elementary operations
# ---------------------------------------------------------------------------
def rows_to_c8(x):
    """Codes int8 and float32 scales of every row of x."""
    v = x.float()
    top = v.abs().amax(1)
    live = top > 0
    full = torch.full_like(top, 127.0)      # (a Python number would be divided through its reciprocal)
    inv = torch.where(live, full / top, torch.zeros_like(top))
    codes = torch.round(v * inv[:, None]).clamp_(-127, 127).to(torch.int8)
    return codes, torch.where(live, top / full, torch.zeros_like(top))


def groups_to_c8(x):
    """Codes int8 [M, C] and the bytes e + 127, uint8 [M, ceil(C / 32)]."""
    M, C = x.shape
    G = -(-C // GROUP)
    v = torch.nn.functional.pad(x.float(), (0, G * GROUP - C)).view(M, G, GROUP)
    top = v.abs().amax(2)
    m, p = torch.frexp(top)                               # top = m 2^p, 1/2 <= m < 1
    e = torch.where(m * 128 <= 127, p - 7, p - 6).clamp_(-126, 122)
    codes = torch.round(torch.ldexp(v, -e[:, :, None]))
    codes = torch.where(codes == 0, torch.sign(v), codes).to(torch.int8)
    return codes.view(M, G * GROUP)[:, :C].contiguous(), (e + 127).to(torch.uint8)


def c8_groups_to(codes, scales, dtype):
    M, C = codes.shape
    e = scales.to(torch.int32).repeat_interleave(GROUP, 1)[:, :C] - 127
    return torch.ldexp(codes.to(dtype), e)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    dt, M = _type(case), case["M"]
    st = dict(case=dict(case), dt=dt)
    if case["op"] == "ckpt":
        # a residual stream: a few columns far above the rest
        x = normal(M, case["C"])
        x[:, :: 97] *= 8.0
        return dict(st, x=x.to(dt))
    if case["op"] == "actbwd":
        codes, scales = groups_to_c8(normal(M, case["C"]).to(dt))
        return dict(st, dy=normal(M, case["C"]).to(dt), z_codes=codes, z_scales=scales)

    K, N, r = case["K"], case["N"], case["r"]
    W = normal(N, K, std=0.02)
    if case["fmt"] == "w8":
        codes, scales = rows_to_c8(W)                     # one scale per output channel
    else:
        v = W.view(N, K // W4_GROUP, W4_GROUP)
        scales = (v.abs().amax(2) / 7.0).half()
        q = torch.round(v * (1.0 / scales.float())[:, :, None]).clamp_(-7, 7).to(torch.int32).view(N, K // 2, 2)
        codes = ((q[:, :, 0] & 15) | ((q[:, :, 1] & 15) << 4)).to(torch.uint8)
        scales = scales.contiguous()
    st.update(codes=codes, scales=scales, alpha=16.0, A=normal(K, r, std=0.05), B=normal(r, N, std=0.05))
    x = normal(M, K).to(dt)
    if case["op"] == "fwd":
        st.update(x=x)
    else:
        xc, xs = rows_to_c8(x)
        st.update(x_codes=xc, x_scales=xs, t=(x.double() @ st["A"].double()).float())
    if case["op"] == "bwd":
        st.update(dy=normal(M, N).to(dt))
        if case["act"] != "none":
            st["z_codes"], st["z_scales"] = groups_to_c8(normal(M, K).to(dt))
        if case["add"]:
            st.update(add=normal(M, K).to(dt))
    else:
        if case["bias"]:
            st.update(bias=normal(N, std=0.1))
        if case["residual"]:
            st.update(residual=normal(M, N).to(dt))
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def act_of(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def slope_of(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        h = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + h) + 0.5 * z * (1.0 - h * h) * c * (1.0 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def weight_of(st, dtype):
    """The dequantized weight [N, K]."""
    if st["case"]["fmt"] == "w8":
        return st["codes"].to(dtype) * st["scales"].to(dtype)[:, None]
    c = st["codes"].to(torch.int32)
    q = torch.stack((c & 15, c >> 4), 2)
    q = torch.where(q > 7, q - 16, q).view(c.shape[0], -1, W4_GROUP).to(dtype)
    return (q * st["scales"].to(dtype)[:, :, None]).reshape(c.shape[0], -1)


def run(st):
    if own:
        return _run_own(st)
    case, dt, op = st["case"], st["dt"], st["case"]["op"]
    if op == "ckpt":
        if case["cfmt"] == "c8row":
            codes, scales = rows_to_c8(st["x"])
            return (codes.float() * scales[:, None]).to(dt)
        return c8_groups_to(*groups_to_c8(st["x"]), torch.float32).to(dt)
    if op == "actbwd":
        dz = st["dy"].float() * slope_of(case["act"], c8_groups_to(st["z_codes"], st["z_scales"], torch.float32))
        return dict(dz=dz.to(dt), dbias=dz.sum(0))
    s = st["alpha"] / case["r"]
    W = weight_of(st, torch.float32)
    if op == "bwd":
        dy = st["dy"].float()
        u = dy @ st["B"].T
        dx = dy @ W + s * (u @ st["A"].T)
        if case["act"] != "none":
            dx = dx * slope_of(case["act"], c8_groups_to(st["z_codes"], st["z_scales"], torch.float32))
        if case["add"]:
            dx = dx + st["add"].float()
        return dict(dx=dx.to(dt), dA=s * (st["x_codes"].float().T @ (u * st["x_scales"][:, None])), dB=s * (st["t"].T @ dy))
    out = {}
    if op == "fwd":
        t = st["x"].float() @ st["A"]
        if case["fmt"] == "w8" or case["save_x"]:
            xc, xs = rows_to_c8(st["x"])
        if case["save_x"]:
            out.update(x_codes=xc, x_scales=xs)
        out.update(t=t)
    else:
        t, xc, xs = st["t"], st["x_codes"], st["x_scales"]
    if case["fmt"] == "w8" or op == "refwd":
        z = (xc.float() @ W.T) * xs[:, None]
    else:
        z = st["x"].float() @ W.T
    z = z + s * (t @ st["B"])
    if case["bias"]:
        z = z + st["bias"]
    if case["save_z"] == "full":
        out.update(z=z.to(dt))
    elif case["save_z"] == "c8g32":
        out.update(z=c8_groups_to(*groups_to_c8(z), torch.float32).to(dt))
    y = act_of(case["act"], z)
    if case["residual"]:
        y = y + st["residual"].float()
    return dict(out, y=y.to(dt))


def _run_own(st):
    from quantized_frozen_weight_amd import binding as Q
    case, dt, op = st["case"], st["dt"], st["case"]["op"]
    if op == "ckpt":
        return Q.qlora_ckpt_read(Q.qlora_ckpt_write(st["x"], case["cfmt"]), dt)
    zc = Q.Checkpoint(st["z_codes"], st["z_scales"], "c8g32") if "z_codes" in st else None
    if op == "actbwd":
        dz, dbias = Q.qlora_act_bwd(case["act"], st["dy"], zc)
        return dict(dz=dz, dbias=dbias)
    lin = Q.QLinear(case["K"], case["N"], case["r"], st["alpha"], case["fmt"], st["codes"], st["scales"], st["A"], st["B"])
    if op == "bwd":
        xc = Q.Checkpoint(st["x_codes"], st["x_scales"], "c8row")
        dx, dA, dB = Q.qlora_bwd_epi(lin, xc, st["dy"], st["t"], act=case["act"], z=zc, add=st.get("add"))
        return dict(dx=dx, dA=dA, dB=dB)
    save_z = None if case["save_z"] == "none" else case["save_z"]
    epilogue = dict(act=case["act"], bias=st.get("bias"), residual=st.get("residual"), save_z=save_z)
    out = {}
    if op == "fwd":
        y, t, z, xc = Q.qlora_fwd_epi(lin, st["x"], save_x=case["save_x"], **epilogue)
        out.update(t=t)
        if xc is not None:
            out.update(x_codes=xc.codes, x_scales=xc.scales)
    else:
        xc = Q.Checkpoint(st["x_codes"], st["x_scales"], "c8row")
        y, z = Q.qlora_fwd_ckpt(lin, xc, st["t"], dt, **epilogue)
    if z is not None:
        # what the group checkpoint stands for
        out.update(z=Q.qlora_ckpt_read(z, dt) if save_z == "c8g32" else z)
    return dict(out, y=y)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    if case["op"] == "ckpt":
        v = st["x"].to(d)
        if case["cfmt"] == "c8row":
            # the code is defined by float32 operations, the value is exact
            top = st["x"].float().abs().max(1, keepdim=True).values
            q = (st["x"].float() * (127.0 / top.to(d)).float()).round()
            return q.to(d) * (top.to(d) / 127.0).float().to(d)
        M, C = v.shape
        pad = -C % GROUP
        v = torch.cat((v, v.new_zeros(M, pad)), 1).reshape(M, -1, GROUP)
        top = v.abs().max(2, keepdim=True).values.clamp(min=2.0 ** -120)
        unit = torch.exp2(torch.ceil(torch.log2(top / 127.0)))
        return (v.sign() * (v / unit).round().abs().clamp(min=1) * unit).reshape(M, -1)[:, :C]

    def groups(codes, scales):
        return torch.stack([codes[:, i].to(d) * torch.exp2(scales[:, i // GROUP].to(d) - 127) for i in range(codes.shape[1])], 1)

    def phi(z):
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))

    def tanh_arg(z):
        return math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)

    f = {"none": lambda z: z, "relu": torch.relu, "gelu": lambda z: z * phi(z),
         "gelu_tanh": lambda z: z * torch.sigmoid(2 * tanh_arg(z)), "silu": lambda z: z * torch.sigmoid(z)}[case["act"]]

    def slope(z):
        with torch.enable_grad():
            z = z.clone().requires_grad_(True)
            return torch.autograd.grad(f(z).sum(), z)[0]

    if case["op"] == "actbwd":
        dz = st["dy"].to(d) * slope(groups(st["z_codes"], st["z_scales"]))
        return dict(dz=dz, dbias=dz.sum(0))
    s, A, B = st["alpha"] / case["r"], st["A"].to(d), st["B"].to(d)
    if case["fmt"] == "w8":
        W = (st["codes"].to(d).T * st["scales"].to(d)).contiguous()
    else:
        c = st["codes"].to(torch.int16)
        nib = lambda v: torch.remainder(v + 8, 16) - 8  # noqa: E731
        q = torch.empty(c.shape[0], 2 * c.shape[1], dtype=d, device=c.device)
        q[:, 0::2], q[:, 1::2] = nib(c % 16).to(d), nib(c // 16).to(d)
        W = (q * st["scales"].to(d).repeat_interleave(W4_GROUP, 1)).T.contiguous()
    if case["op"] == "bwd":
        dy = st["dy"].to(d)
        u = dy @ B.T.contiguous()
        dx = dy @ W.T.contiguous() + s * (u @ A.T.contiguous())
        if case["act"] != "none":
            dx = dx * slope(groups(st["z_codes"], st["z_scales"]))
        if case["add"]:
            dx = dx + st["add"].to(d)
        x = st["x_codes"].to(d) * st["x_scales"].to(d)[:, None]
        return dict(dx=dx, dA=s * (x.T.contiguous() @ u), dB=s * (st["t"].to(d).T.contiguous() @ dy))
    out = {}
    if case["op"] == "fwd":
        x = st["x"].to(d)
        t = x @ A
        top = st["x"].float().abs().max(1, keepdim=True).values
        codes = (st["x"].float() * (127.0 / top.to(d)).float()).round()
        unit = (top.to(d) / 127.0).float().to(d)
        if case["save_x"]:
            out.update(x_codes=None, x_scales=unit[:, 0])
        if case["fmt"] == "w8":
            x = codes.to(d) * unit
        out.update(t=t)
    else:
        x, t = st["x_codes"].to(d) * st["x_scales"].to(d)[:, None], st["t"].to(d)
    z = x @ W + s * (t @ B)
    if case["bias"]:
        z = z + st["bias"].to(d)
    if case["save_z"] != "none":
        # a group checkpoint's codes are defined from z in 32 bits
        out.update(z=z if case["save_z"] == "full" else None)
    y = f(z)
    if case["residual"]:
        y = y + st["residual"].to(d)
    return dict(out, y=y)
