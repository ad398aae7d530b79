"""What the vocabulary layer and the adapter optimizer of libqlora cost.

A vocabulary layer is a frozen quantized W [K, N] (column v: the K features of
vocabulary entry v; entries from ``vocab`` to N, the next multiple of 16, are
padding) with an optional float32 adapter A [K, r], B [r, N], s = alpha / r:
its columns w_v = deq(W)[:, v] + s A B[:, v] are the embedding of token v at
the model's input and the classifier of token v at its output. The operators:

* ``embed``     x[m] = scale w_token(m), a row of zeros for a token that is not
                in [0, vocab);
* ``embedbwd``  dA and dB of that for the gradient dy of x: dB by the tokens'
                rows, dA over all of them;
* ``loss``      the softmax cross entropy of the logits l[m, v] = xq[m] . w_v
                with x quantized to 8 bits by rows as in the layer's forward:
                loss[m] = lse[m] - l[m, target(m)], lse[m] the logarithm of
                sum_v exp(l[m, v]); 0 for a target that is not in [0, vocab);
* ``train``     the same, then its gradient: dl[m, v] = dloss[m] (exp(l[m, v] -
                lse[m]) - [v = target(m)]), u = dl B^T, dx = dl deq(W)^T +
                s u A^T, dA = s x^T u, dB = s (x A)^T dl;
* ``adamw``     one AdamW step of many float32 tensors with the gradient's
                global norm clipped, the moments in 32 or in 8 bits.

8-bit moments ("s8"): 32 consecutive elements of a tensor share the scale 2^e,
kept as the byte e + 127. The first moment's byte is a sign, 3 bits of exponent
and 4 of mantissa, the root of the second moment's 3 bits of exponent and 5 of
mantissa (exponent 0: subnormal; the largest 31/16 and 63/32, and e the
smallest, at least -126, that covers the group). They are rounded up where the low bits of
hash(tensor, element, step, seed) say so, as often as the value is nearer the
upper code, so that moves far below a code's step are not lost; a second moment
that is not 0 keeps a code that is not 0.
"""

import math

import torch

own = False

W4_GROUP = 128                  # inputs per scale of a 4-bit weight
S8_GROUP = 32                   # elements per scale of an 8-bit moment
IGNORED = -100                  # the target of a row that has none


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the tokens of one small batch: all latency
        dict(name="embed f32 64x256 v4096", op="embed", fmt="w8", dtype="f32", M=64, K=256, vocab=4096, r=4,
             itype="i64"),
        # 16 sequences of 512 tokens into a 2048-wide decoder with a large vocabulary
        dict(name="embed 8192x2048 v256000", op="embed", fmt="w8", dtype="bf16", M=8192, K=2048, vocab=256000, r=8,
             itype="i64"),
        # a ragged batch at the width of a small transformer, odd vocabulary
        dict(name="embedbwd 1001x768 v50257", op="embedbwd", fmt="w8", dtype="bf16", M=1001, K=768, vocab=50257, r=4,
             itype="i64"),
        # the gradient of the 8192 tokens
        dict(name="embedbwd 8192x2048 v256000", op="embedbwd", fmt="w8", dtype="bf16", M=8192, K=2048, vocab=256000,
             r=8, itype="i32"),
        # the score of one token (serving)
        dict(name="loss 1x2048 v256000", op="loss", fmt="w8", dtype="bf16", M=1, K=2048, vocab=256000, r=0,
             itype="i64"),
        # 32 sequences of 128 tokens, validation
        dict(name="loss 4096x768 v50257", op="loss", fmt="w8", dtype="bf16", M=4096, K=768, vocab=50257, r=4,
             itype="i64"),
        # a small float32 classifier, odd sizes
        dict(name="train f32 77x256 v1000", op="train", fmt="w8", dtype="f32", M=77, K=256, vocab=1000, r=4,
             itype="i64"),
        # four sequences of 512 tokens, large frozen vocabulary
        dict(name="train 2048x2048 v256000", op="train", fmt="w8", dtype="bf16", M=2048, K=2048, vocab=256000, r=0,
             itype="i64"),
        # a batch through an adapted, tied vocabulary
        dict(name="train 4096x768 v50257 r8", op="train", fmt="w8", dtype="bf16", M=4096, K=768, vocab=50257, r=8,
             itype="i64"),
        # the 4-bit vocabulary of a 4096-wide model
        dict(name="train w4 1024x4096 v32000", op="train", fmt="w4g128", dtype="bf16", M=1024, K=4096, vocab=32000, r=0,
             itype="i32"),
        # the adapter of one layer: all latency
        dict(name="adamw f32 2 tensors", op="adamw", state="f32", tensors=2, least=1024, most=1024, clip=1.0),
        # every adapter of a decoder's projections and feed-forward layers, rank 32 to 64
        dict(name="adamw s8 56 tensors", op="adamw", state="s8", tensors=56, least=65536, most=1048576, clip=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_MACS = 2048 * 2048 * 256000        # the largest listed product
MOST_LOGITS = 2048 * 256000


def draw(rng):
    op = rng.choice(["embed", "embedbwd", "loss", "train", "train", "adamw"])
    if op == "adamw":
        tensors = _log(rng, 1, 60)
        most = _log(rng, 8, (1 << 24) // tensors)
        return dict(op=op, state=rng.choice(["f32", "s8"]), tensors=tensors, least=max(1, most // rng.choice([1, 7, 64])),
                    most=most, clip=rng.choice([0.0, 1.0, 1.0]))
    f32 = rng.random() < 0.25
    fmt = "w8" if f32 else rng.choice(["w8", "w8", "w4g128"])
    unit = 128 if fmt == "w4g128" else 16
    K = unit * _log(rng, 1, (1024 if f32 else 4096) // unit)
    vocab = _log(rng, 16, 262144)
    M = _log(rng, 1, 8192)
    r = rng.choice([0, 0, 1, 3, 4, 8, 16, 32])
    if op in ("embed", "embedbwd"):
        M = max(1, min(M, 8192 * 2048 // K))
        r = max(r, 1) if op == "embedbwd" else r
    else:
        M = max(1, min(M, MOST_MACS // (K * vocab), MOST_LOGITS // vocab))
    return dict(op=op, fmt=fmt, dtype="f32" if f32 else "bf16", M=M, K=K, vocab=vocab, r=r,
                itype=rng.choice(["i32", "i64"]))


def padded(vocab):
    return -(-vocab // 16) * 16


def work(case):
    if case["op"] == "adamw":
        n = sum(sizes(case))
        moments = 16 if case["state"] == "f32" else 4 + 4 / S8_GROUP
        return dict(bytes=n * (12 + moments), flops=n * (22 if case["clip"] else 20))
    e = 4 if case["dtype"] == "f32" else 2
    M, K, V, r = case["M"], case["K"], case["vocab"], case["r"]
    row = K + 4 if case["fmt"] == "w8" else K // 2 + 2 * (K // W4_GROUP)      # one vocabulary entry
    ids = M * (4 if case["itype"] == "i32" else 8)
    N = padded(V)
    if case["op"] == "embed":
        return dict(bytes=ids + M * (e * K + row) + 4 * r * (K + M), flops=M * K * (2 + 2 * r))
    if case["op"] == "embedbwd":
        return dict(bytes=ids + e * M * K + 4 * r * (2 * K + M + N), flops=4 * M * K * r)
    product = 2 * M * K * V + 2 * M * r * (K + V)
    b = ids + row * V + e * M * K + 4 * r * (K + V) + 8 * M
    if case["op"] == "loss":
        return dict(bytes=b + 4 * M * r, flops=product)
    return dict(bytes=b + 4 * M + e * M * K + 4 * r * (K + N), flops=2 * product + 4 * M * r * (K + V))


# ---------------------------------------------------------------------------
# quantized forms in elementary operations
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


def hashed(where, step, seed):
    """32 bits of hash for every element, as int64: two rounds of multiply and
    shift over where (the tensor's and the element's number) and the step."""
    low = 0xFFFFFFFF
    x = (where + (step.to(torch.int64) * 0xBB67AE85 + seed)) & low
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & low
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & low
    return x ^ (x >> 16)


def to_s8(v, random, mantissa):
    """Codes of |v| (3 bits of exponent over `mantissa` bits) and bytes e + 127;
    `random`: 16 bits an element."""
    g = v.abs().view(-1, S8_GROUP)
    top = g.amax(1)
    m, p = torch.frexp(top)                                # top = m 2^p, 1/2 <= m < 1
    e = torch.where(m > 1 - 2.0 ** -(mantissa + 1), p, p - 1)
    e = torch.where(top > 0, e, torch.full_like(e, -126)).clamp_(-126, 127)
    # 7 steps of exponent under the group's scale: the code is the top of a
    # float32 whose exponent field is the code's
    f = torch.ldexp(torch.ldexp(g, -e[:, None]), torch.full_like(e, -120)[:, None])
    shift = 23 - mantissa
    bits = f.contiguous().view(torch.int32) + (random.view(-1, S8_GROUP) << (shift - 16))
    return (bits >> shift).view(-1), (e + 127).to(torch.uint8)


def of_s8(codes, scales, mantissa):
    f = (codes.to(torch.int32) << (23 - mantissa)).view(torch.float32)
    e = scales.to(torch.int32).repeat_interleave(S8_GROUP) - 127
    return torch.ldexp(torch.ldexp(f, torch.full_like(e, 120)), e)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def sizes(case):
    """Elements of every tensor: the ranges' ends and what lies between them,
    every third an odd number."""
    n, lo, hi = case["tensors"], case["least"], case["most"]
    mid = [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]
    return [max(1, k - (i % 3 == 2)) for i, k in enumerate(mid)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    st = dict(case=dict(case))
    if case["op"] == "adamw":
        # one buffer a kind, every tensor a slice of it that begins at a group
        n = sizes(case)
        start = [0]
        for k in n:
            start.append(start[-1] + -(-k // S8_GROUP) * S8_GROUP)
        total = start[-1]
        item = torch.repeat_interleave(torch.arange(len(n), device="cuda"),
                                       torch.tensor([b - a for a, b in zip(start, start[1:])], device="cuda"))
        inside = torch.arange(total, device="cuda") - torch.tensor(start[:-1], device="cuda")[item]
        live = (inside < torch.tensor(n, device="cuda")[item]).float()
        low = 0xFFFFFFFF
        st.update(lr=5e-5, betas=(0.9, 0.999), eps=1e-6, clip=case["clip"], seed=seed & 0xFFFF, n=n, start=start, live=live,
                  # biases and the like are not decayed
                  decay=[0.0 if i % 4 == 3 else 0.01 for i in range(len(n))],
                  where=((inside * 0x9E3779B1) & low) + ((item * 0x3C6EF373) & low),
                  step=torch.full((1,), 9, dtype=torch.int32, device="cuda"), p=normal(total, std=0.05) * live,
                  # gradients of elements of very different size
                  g=normal(total, std=1e-3) * torch.exp(normal(total)) * live)
        st["wd"] = torch.tensor(st["decay"], device="cuda")[item]
        m, v = 0.3 * normal(total, std=1e-3) * live, (1e-3 * torch.exp(normal(total))) ** 2 * (1e-2 * live)
        if case["state"] == "f32":
            st.update(m=m, v=v)
        else:
            half = torch.full((total,), 1 << 15, dtype=torch.int32, device="cuda")
            c, st["m_scales"] = to_s8(m, half, 4)
            st["m"] = (c + 128 * (m < 0)).to(torch.uint8)
            c, st["v_scales"] = to_s8(torch.sqrt(v), half, 5)
            st["v"] = torch.where((c == 0) & (v > 0), torch.ones_like(c), c).to(torch.uint8)
        return st

    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    M, K, V, r = case["M"], case["K"], case["vocab"], case["r"]
    N = padded(V)
    st.update(dt=dt, N=N, alpha=16.0, scale=math.sqrt(K), A=None, B=None)
    W = normal(N, K, std=0.02)
    W[V:] = 0
    if case["fmt"] == "w8":
        st["codes"], st["scales"] = rows_to_c8(W)            # one scale per vocabulary entry
    else:
        v = W.view(N, K // W4_GROUP, W4_GROUP)
        scales = (v.abs().amax(2) / 7.0).half()
        inv = torch.where(scales > 0, 1.0 / scales.float(), torch.zeros_like(scales, dtype=torch.float32))
        q = torch.round(v * inv[:, :, None]).clamp_(-7, 7).to(torch.int32).view(N, K // 2, 2)
        st["codes"] = ((q[:, :, 0] & 15) | ((q[:, :, 1] & 15) << 4)).to(torch.uint8)
        st["scales"] = scales.contiguous()
    if r:
        st.update(A=normal(K, r, std=0.05), B=normal(r, N, std=0.05))
    # tokens as in text: the rank of a token over its frequency
    ids = (torch.exp(uniform(M) * math.log(V + 1.0)) - 1).to(torch.int64).clamp_(0, V - 1)
    it = torch.int32 if case["itype"] == "i32" else torch.int64
    if case["op"] in ("embed", "embedbwd"):
        ids = torch.where(uniform(M) < 0.03, torch.full_like(ids, -1), ids)          # padding
        st.update(tokens=ids.to(it))
        return dict(st, dy=normal(M, K).to(dt)) if case["op"] == "embedbwd" else st
    # half of the rows lean to their target, as a trained model's do
    x = normal(M, K)
    lean = 8.0 * (uniform(M) < 0.5).float()
    x = x + lean[:, None] * W[ids] / (0.02 * math.sqrt(K))
    ids = torch.where(uniform(M) < 0.1, torch.full_like(ids, IGNORED), ids)           # prompts and padding
    st.update(x=x.to(dt), targets=ids.to(it))
    if case["op"] == "train":
        st["dloss"] = torch.ones(M, device="cuda") / (ids >= 0).sum().clamp(min=1)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
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
    case, op = st["case"], st["case"]["op"]
    if op == "adamw":
        return _adamw_plain(st)
    dt, r, V = st["dt"], case["r"], case["vocab"]
    s = st["alpha"] / r if r else 0.0
    if op in ("embed", "embedbwd"):
        ids = st["tokens"].to(torch.int64)
        ok = (ids >= 0) & (ids < V)
        at = torch.where(ok, ids, torch.zeros_like(ids))
        if op == "embedbwd":
            dy = st["dy"].float() * (st["scale"] * s * ok.float())[:, None]
            dB = torch.zeros(st["N"], r, device=dy.device).index_add_(0, at, dy @ st["A"])
            return dict(dA=dy.T @ st["B"].T[at], dB=dB.T.contiguous())
        rows = dict(st, codes=st["codes"][at], scales=st["scales"][at])
        x = weight_of(rows, torch.float32)
        if r:
            x = x + s * (st["B"].T[at] @ st["A"].T)
        return (torch.where(ok[:, None], st["scale"] * x, torch.zeros_like(x))).to(dt)
    W = weight_of(st, torch.float32)[:V]
    x, ids = st["x"].float(), st["targets"].to(torch.int64)
    ok = (ids >= 0) & (ids < V)
    at = torch.where(ok, ids, torch.zeros_like(ids))
    xc, xs = rows_to_c8(x)
    logits = (xc.float() @ W.T) * xs[:, None]
    out = {}
    if r:
        t = x @ st["A"]
        logits += s * (t @ st["B"][:, :V])
        out.update(t=t)
    top = logits.amax(1)
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
    loss = torch.where(ok, lse - logits.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    out.update(loss=loss, lse=lse)
    if op == "loss":
        return out
    dl = torch.exp(logits - lse[:, None])
    del logits
    dl.scatter_add_(1, at[:, None], torch.full_like(lse, -1.0)[:, None])
    dl *= (st["dloss"] * ok.float())[:, None]
    dx = dl @ W
    if r:
        u = dl @ st["B"][:, :V].T
        dx += s * (u @ st["A"].T)
        dB = torch.zeros_like(st["B"])
        dB[:, :V] = s * (t.T @ dl)
        out.update(dA=s * (x.T @ u), dB=dB)
    return dict(out, dx=dx.to(dt))


def _adamw_plain(st):
    b1, b2 = st["betas"]
    g, eight = st["g"], st["case"]["state"] == "s8"
    norm = torch.sqrt(g.double().square().sum()).float()
    if st["clip"]:
        g = g * (st["clip"] / torch.clamp(norm, min=st["clip"]))
    st["step"] += 1
    step = st["step"].double()
    c1, c2 = (1 - b1 ** step).float(), (1 - b2 ** step).float()
    if eight:
        sign = 1.0 - 2.0 * (st["m"] >> 7).float()
        m, v = sign * of_s8(st["m"] & 127, st["m_scales"], 4), of_s8(st["v"], st["v_scales"], 5).square()
    else:
        m, v = st["m"], st["v"]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * (g * g)
    root = torch.sqrt(v)
    st["p"] *= 1 - st["lr"] * st["wd"]
    st["p"] -= (st["lr"] / c1) * (m / (root / torch.sqrt(c2) + st["eps"]))
    if not eight:
        st["m"].copy_(m)
        st["v"].copy_(v)
        return dict(p=st["p"], m=m, v=v, norm=norm, step=st["step"])
    h = hashed(st["where"], st["step"], st["seed"]).to(torch.int32)
    c, scales = to_s8(m, h & 0xFFFF, 4)
    st["m"].copy_(c + 128 * (m < 0))
    st["m_scales"].copy_(scales)
    c, scales = to_s8(root, (h >> 16) & 0xFFFF, 5)
    st["v"].copy_(torch.where((c == 0) & (root > 0), torch.ones_like(c), c))
    st["v_scales"].copy_(scales)
    return dict(p=st["p"], norm=norm, step=st["step"], **_moments(st))


def _moments(st):
    """What the 8-bit moments stand for: the first, and the second's root."""
    sign = 1.0 - 2.0 * (st["m"] >> 7).float()
    return dict(m=(sign * of_s8(st["m"] & 127, st["m_scales"], 4)).bfloat16(),
                root_v=of_s8(st["v"], st["v_scales"], 5).bfloat16())


def _run_own(st):
    from quantized_frozen_weight_amd import binding as Q
    case, op = st["case"], st["case"]["op"]
    if op == "adamw":
        eight = case["state"] == "s8"
        if "optimizer" not in st:
            # the program's optimizer, over tensors that it holds
            def parts(t, unit=1):
                return [t[a // unit: a // unit + -(-n // unit)] for a, n in zip(st["start"], st["n"])]

            st["optimizer"] = Q.AdamW(
                parts(st["p"]), state=case["state"], decay=st["decay"], step=st["step"], m=parts(st["m"]), v=parts(st["v"]),
                m_scales=parts(st["m_scales"], S8_GROUP) if eight else None,
                v_scales=parts(st["v_scales"], S8_GROUP) if eight else None, seed=st["seed"])
            st["grads"] = parts(st["g"])
        norm = Q.qlora_adamw(st["optimizer"], st["grads"], lr=st["lr"], betas=st["betas"], eps=st["eps"],
                             clip_norm=st["clip"], need_norm=True)
        moments = dict(m=st["m"], v=st["v"])
        if eight:
            # what the codes stand for, as a program that looks at its state reads it
            moments = dict(m=Q.qlora_moment_read(st["m"], st["m_scales"], "m", torch.bfloat16),
                           root_v=Q.qlora_moment_read(st["v"], st["v_scales"], "root_v", torch.bfloat16))
        return dict(p=st["p"], norm=norm.reshape(()), step=st["step"], **moments)
    layer = Q.QLinear(case["K"], st["N"], case["r"], st["alpha"], case["fmt"], st["codes"], st["scales"], st["A"], st["B"])
    V = case["vocab"]
    if op == "embed":
        return Q.qlora_embed(layer, st["tokens"], vocab=V, scale=st["scale"], dtype=st["dt"])
    if op == "embedbwd":
        dA, dB = Q.qlora_embed_bwd(layer, st["tokens"], st["dy"], vocab=V, scale=st["scale"])
        return dict(dA=dA, dB=dB)
    loss, lse, t = Q.qlora_xent_fwd(layer, st["x"], st["targets"], vocab=V)
    out = dict(loss=loss, lse=lse)
    if case["r"]:
        out.update(t=t)
    if op == "loss":
        return out
    dx, dA, dB = Q.qlora_xent_bwd(layer, st["x"], st["targets"], lse, st["dloss"], t=t, vocab=V)
    if case["r"]:
        out.update(dA=dA, dB=dB)
    return dict(out, dx=dx)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    if case["op"] == "adamw":
        b1, b2 = st["betas"]
        g = st["g"].to(d)
        norm = torch.linalg.vector_norm(g)
        if case["clip"]:
            g = g * min(1.0, case["clip"] / max(float(norm), 1e-300))
        if case["state"] == "f32":
            m, v = st["m"].to(d), st["v"].to(d)
        else:
            def value(codes, bits, scales):
                ex, man = codes >> bits, codes & ((1 << bits) - 1)
                f = torch.where(ex > 0, 1 + man.to(d) / 2 ** bits, man.to(d) / 2 ** bits)
                f = f * torch.exp2(ex.clamp(min=1).to(d) - 7)
                return f * torch.exp2(scales.to(d) - 127).repeat_interleave(S8_GROUP)

            c = st["m"].long()
            m = value(c % 128, 4, st["m_scales"]) * torch.where(c >= 128, -1.0, 1.0)
            v = value(st["v"].long(), 5, st["v_scales"]) ** 2
        t = int(st["step"]) + 1
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g ** 2
        p = st["p"].to(d) * (1 - st["lr"] * st["wd"].to(d))
        p = p - st["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + st["eps"])
        if case["state"] == "f32":
            return dict(p=p, m=m, v=v, norm=norm, step=None)
        # (the codes come from a hash of the element: no value in 64 bits)
        return dict(p=p, m=None, root_v=None, norm=norm, step=None)
    K, V, r = case["K"], case["vocab"], case["r"]
    s = st["alpha"] / r if r else 0.0
    if case["fmt"] == "w8":
        W = st["codes"].to(d) * st["scales"].to(d)[:, None]
    else:
        c = st["codes"].to(torch.int16)
        nib = lambda v: torch.remainder(v + 8, 16) - 8  # noqa: E731
        W = torch.empty(c.shape[0], K, dtype=d, device=c.device)
        W[:, 0::2], W[:, 1::2] = nib(c % 16).to(d), nib(c // 16).to(d)
        W *= st["scales"].to(d).repeat_interleave(W4_GROUP, 1)
    if r:
        A, B = st["A"].to(d), st["B"].to(d)
    if case["op"] in ("embed", "embedbwd"):
        ids = st["tokens"].long()
        rows = ((ids >= 0) & (ids < V)).nonzero()[:, 0]
        tok = ids[rows]
        if case["op"] == "embed":
            x = torch.zeros(case["M"], K, dtype=d, device=W.device)
            x[rows] = st["scale"] * (W[tok] + (s * (B.T[tok].contiguous() @ A.T.contiguous()) if r else 0))
            return x
        dy = st["scale"] * s * st["dy"][rows].to(d)
        # rows of one token are a run of the sorted tokens: differences of running sums
        order = torch.argsort(tok, stable=True)
        run = torch.cat((torch.zeros(1, r, dtype=d, device=dy.device), (dy @ A)[order].cumsum(0)))
        ends = torch.searchsorted(tok[order].contiguous(), torch.arange(st["N"] + 1, device=dy.device))
        dB = (run[ends[1:]] - run[ends[:-1]]).T
        return dict(dA=dy.T.contiguous() @ B.T[tok].contiguous(), dB=dB)
    x, ids = st["x"].to(d), st["targets"].long()
    top = st["x"].float().abs().max(1, keepdim=True).values
    codes = (st["x"].float() * (127.0 / top.to(d)).float()).round()
    logits = (codes.to(d) * (top.to(d) / 127.0).float().to(d)) @ W[:V].T.contiguous()
    out = {}
    if r:
        t = x @ A
        logits += s * (t @ B[:, :V].contiguous())
        out.update(t=t)
    lse = torch.logsumexp(logits, 1)
    rows = ((ids >= 0) & (ids < V)).nonzero()[:, 0]
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - logits[rows, ids[rows]]
    out.update(loss=loss, lse=lse)
    if case["op"] == "loss":
        return out
    dl = logits.sub_(lse[:, None]).exp_()
    dl[rows, ids[rows]] -= 1
    keep = torch.zeros_like(lse)
    keep[rows] = st["dloss"].to(d)[rows]
    dl *= keep[:, None]
    dx = dl @ W[:V]
    if r:
        u = dl @ B[:, :V].T.contiguous()
        dx += s * (u @ A.T.contiguous())
        dB = torch.zeros_like(B)
        dB[:, :V] = s * (t.T.contiguous() @ dl)
        out.update(dA=s * (x.T.contiguous() @ u), dB=dB)
    return dict(out, dx=dx)
