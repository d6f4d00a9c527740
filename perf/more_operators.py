"""Cases of the operators that finish a training step beside the matrix
optimizers: the AdamW step over a list of tensors (embeddings, heads, norms,
biases), with its two states in 32 or in 8 bits, and the softmax cross entropy
of an output head, which takes the head's product with it and never keeps the
logits.

``run`` computes an operator in its plain form (elementary torch operations in
float32, rounded once) or, where ``own`` is true, through
``rank_orthonormalized_optimizer_dion_amd``.  ``exact`` computes the same
outputs from the definitions in float64.

Formulas:
  AdamW          g = c G;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
                 X = (1 - lr wd) X - lr / (1 - b1^t) m /
                     (sqrt(v) / sqrt(1 - b2^t) + eps).
  8-bit states   m and s = sqrt(v) in blocks of 64 elements: e4m3 values times
                 one power of two per block (a byte e for 2^(e - 127), e8m0):
                 the exponent byte of the block's largest magnitude less 7, at
                 least 1.  A scaled magnitude a becomes floor(a / ulp + u) ulp,
                 ulp = 2^(max(floor(log2 a), -6) - 3), where u has 16 bits of a
                 hash of the element's index and the caller's seed; a nonzero s
                 takes at least one ulp.
  cross entropy  z = x W^T;  lse = log sum_j exp z_j;
                 loss = lse - (1 - e) z_y - e mean_j z_j + zc lse^2, zero where
                 y is the ignored index;
                 dz_j = dloss ((1 + 2 zc lse) exp(z_j - lse) - (1 - e) [j = y]
                 - e / n), zero in ignored rows;  dx = dz W;  dW = dz^T x.
"""
import math

import torch

own = False

LR, BETA1, BETA2, EPS, DECAY, STEP, SEED = 1e-3, 0.9, 0.95, 1e-8, 0.1, 100, 7
BLOCK = 64
IGNORE = -100


def listed():
    return [
        # one norm's gain: the call's latency is what a user sees
        _adamw("adamw 768 f32", "one", 768, 0, 1, "f32", 32),
        # norms and biases of 36 layers: 144 short vectors in one call
        _adamw("adamw 144 vectors", "vectors", 768, 0, 144, "f32", 32),
        # a narrow model's embedding with an odd vocabulary, bfloat16 gradients
        _adamw("adamw 50257x768 bf16", "one", 50257, 768, 1, "bf16", 32),
        # embedding and head of a wide model, states in 8 bits
        _adamw("adamw8 2 x 32000x4096 bf16", "same", 32000, 4096, 2, "bf16", 8),
        # odd sizes, states in 8 bits, one tensor whose gradient and states are zero
        _adamw("adamw8 ragged f32", "ragged", 3001, 517, 7, "f32", 8),
        # the score of one token
        _head("loss 1 token", "forward", 1, 768, 32000, "bf16", 0.0, 0.0),
        # a training batch on a wide model's head: the largest forward
        _head("loss 8192 tokens", "forward", 8192, 4096, 32000, "bf16", 0.0, 0.0),
        # odd sizes in float32, with label smoothing and z-loss
        _head("loss ragged f32", "forward", 1021, 773, 50257, "f32", 0.1, 1e-4),
        # gradients of a few tokens (fine-tuning on short answers)
        _head("loss backward 24 tokens", "backward", 24, 2048, 32000, "bf16", 0.0, 0.0),
        # gradients of a batch, narrow model, odd vocabulary
        _head("loss backward 4096 tokens", "backward", 4096, 768, 50257, "bf16", 0.0, 1e-4),
        # gradients of a training batch on a wide model's head: the largest
        _head("loss backward 8192 tokens", "backward", 8192, 4096, 32000, "bf16", 0.0, 0.0),
        # odd sizes in float32, backward, with label smoothing
        _head("loss backward ragged f32", "backward", 515, 517, 10007, "f32", 0.1, 0.0),
    ]


def draw(rng):
    """One more case: an operator, then its sizes over their whole range."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    if rng.random() < 0.4:
        layout = rng.choice(("one", "ragged", "ragged", "vectors"))
        gdt, bits = rng.choice(("f32", "bf16")), rng.choice((32, 8))
        if layout == "vectors":
            return _adamw(None, layout, log_int(1, 20000), 0, log_int(2, 300), gdt, bits)
        return _adamw(None, layout, log_int(1, 8000), log_int(1, 8000), 1 if layout == "one" else rng.randint(2, 9),
                      gdt, bits)
    kind = rng.choice(("forward", "backward"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    tokens, k = log_int(1, 8192), log_int(64, 8192)
    if rng.random() < 0.5:
        k = -(-k // 64) * 64
    # as many columns as keep the call below the largest listed one
    most = 8192 * 4096 * 32000 // (1 if dtype == "bf16" else 4)
    n = log_int(100, max(101, min(140000, most // (tokens * k))))
    return _head(None, kind, tokens, k, n, dtype, rng.choice((0.0, 0.0, 0.1)), rng.choice((0.0, 1e-4)))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "adamw":
        return _prepare_adamw(case, g)
    t, k, n, dt = case["tokens"], case["k"], case["n"], _dtype(case["dtype"])
    # a few words are frequent, most are rare; half of the tokens are predicted well
    y = ((torch.rand(t, generator=g, device="cuda") * math.log(n + 1.0)).exp() - 1.0).long().clamp(0, n - 1)
    w = torch.randn(n, k, generator=g, device="cuda").mul_(2.0 * k ** -0.5)
    sure = 2.0 * (torch.rand(t, 1, generator=g, device="cuda") < 0.5)
    x = torch.randn(t, k, generator=g, device="cuda").addcmul_(w[y], sure)
    y = torch.where(torch.rand(t, generator=g, device="cuda") < 0.1 * (t > 1), IGNORE, y)
    s = {"case": case, "x": x.to(dt), "w": w.to(dt), "y": y}
    if case["op"] == "forward":
        s["loss"], s["lse"] = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
        return s
    s["lse"] = torch.logsumexp(s["x"].float() @ s["w"].float().t(), 1)
    s["dloss"] = torch.rand(t, generator=g, device="cuda").add_(0.5).div_(t)   # weighted mean
    s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
    return s


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "adamw":
        return _adamw_plain(state) if case["bits"] == 32 else _adamw8_plain(state)
    return _forward_plain(state, case) if case["op"] == "forward" else _backward_plain(state, case)


def _run_own(s, case):
    import rank_orthonormalized_optimizer_dion_amd as dion
    if case["op"] == "adamw":
        if "plan" not in s:
            s["plan"] = dion.AdamWPlan(s["list"], weight_decay=s["wd"])
        s["plan"].step(LR, STEP, betas=(BETA1, BETA2), eps=EPS, grad_scale=s["scale"], seed=SEED)
        return _adamw_outputs(s)
    kw = dict(ignore_index=IGNORE, label_smoothing=case["smoothing"], z_loss=case["z_loss"], workspace=s.get("ws"))
    if case["op"] == "forward":
        s["ws"] = dion.cross_entropy_forward(s["x"], s["w"], s["y"], s["loss"], lse=s["lse"], **kw)
        return {"loss": s["loss"], "lse": s["lse"]}
    s["ws"] = dion.cross_entropy_backward(s["dloss"], s["x"], s["w"], s["y"], s["lse"], dx=s["dx"], dw=s["dw"], **kw)
    return {"dx": s["dx"], "dw": s["dw"]}


def work(case):
    if case["op"] == "adamw":
        n = sum(math.prod(s) for s in _shapes(case))
        states = 16 if case["bits"] == 32 else 4 + 4 / BLOCK
        return {"bytes": n * (8 + _size(case["gdt"]) + states), "flops": 15.0 * n}
    t, k, n, e = case["tokens"], case["k"], case["n"], _size(case["dtype"])
    if case["op"] == "forward":
        return {"bytes": (t * k + n * k) * e + 16 * t, "flops": 2.0 * t * k * n}
    # the logits are not kept, so z is computed again
    return {"bytes": 2 * (t * k + n * k) * e + 16 * t, "flops": 6.0 * t * k * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _adamw64(s, case)
    x, w, y = s["x"].double(), s["w"].double(), s["y"]
    n, e, zc = case["n"], case["smoothing"], case["z_loss"]
    z = torch.mm(x, w.t().contiguous())
    taken = y != IGNORE
    if case["op"] == "forward":
        lse = torch.logsumexp(z, 1)
        hit = z.gather(1, y.clamp(min=0)[:, None])[:, 0]
        loss = lse - (1 - e) * hit - e * z.mean(1) + zc * lse.square()
        return {"loss": torch.where(taken, loss, 0.0), "lse": lse}
    # the gradient at the given lse: d/dz of exp(z - lse) forms, not of logsumexp
    lse = s["lse"].double()[:, None]
    dz = torch.exp(z - lse).mul_(1 + 2 * zc * lse).sub_(e / n)
    dz[torch.arange(len(y), device=y.device), y.clamp(min=0)] -= 1 - e
    dz *= (s["dloss"].double() * taken)[:, None]
    return {"dx": torch.mm(dz, w), "dw": torch.mm(dz.t().contiguous(), x)}


# --- cases -------------------------------------------------------------------

def _named(name, case):
    return case if name is None else {"name": name, **case}


def _adamw(name, layout, m, n, count, gdt, bits):
    return _named(name, {"op": "adamw", "layout": layout, "m": m, "n": n, "count": count, "gdt": gdt, "bits": bits})


def _head(name, op, tokens, k, n, dtype, smoothing, z_loss):
    return _named(name, {"op": op, "tokens": tokens, "k": k, "n": n, "dtype": dtype, "smoothing": smoothing,
                         "z_loss": z_loss})


def _shapes(case):
    """The tensors of a step: `count` vectors, `count` matrices of one shape,
    or matrices that shrink by odd steps, each followed by its bias."""
    m, n, count = case["m"], case["n"], case["count"]
    if case["layout"] == "vectors" or n == 0:
        return [(m,)] * count
    if case["layout"] in ("one", "same"):
        return [(m, n)] * count
    sizes = [(max(1, m - 37 * (i // 2)), max(1, n - 11 * (i // 2))) for i in range(count)]
    return [s if i % 2 == 0 else s[:1] for i, s in enumerate(sizes)]


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _size(name):
    return 2 if name == "bf16" else 4


def _prepare_adamw(case, g):
    """Tensors are views of flat buffers, as programs lay them out that reduce
    gradients in buckets: matrices (decayed) first, then vectors, each padded
    with zeros to a whole block."""
    shapes = sorted(_shapes(case), key=len, reverse=True)
    sizes = [math.prod(s) for s in shapes]
    room = [-(-n // BLOCK) * BLOCK for n in sizes]
    starts = [sum(room[:i]) for i in range(len(room))]
    total, decayed = sum(room), sum(r for s, r in zip(shapes, room) if len(s) == 2)
    if len(set(sizes)) == 1:   # one pattern for all
        used = (torch.arange(room[0], device="cuda") < sizes[0]).repeat(len(sizes))
    else:
        used = torch.cat([torch.arange(r, device="cuda") < n for r, n in zip(room, sizes)])

    def normal():
        return torch.randn(total, generator=g, device="cuda")

    # rows of a model's tensors differ in scale by orders of magnitude
    size = normal().view(-1, BLOCK)[:, :1].mul(1.5).exp().mul_(1e-3).expand(-1, BLOCK).reshape(-1)
    zero = 1.0
    if case["layout"] == "ragged":   # an expert that no token took
        zero = torch.ones(total, device="cuda")
        zero[starts[-1]:].zero_()
    s = {"case": case, "shapes": shapes, "sizes": sizes, "room": room, "starts": starts, "decayed": decayed,
         "X": normal().mul_(0.02).mul_(used), "G": (normal() * size * used * zero).to(_dtype(case["gdt"])),
         "scale": torch.rand(1, generator=g, device="cuda").mul_(0.5).add_(0.5),
         "wd": [DECAY if len(x) == 2 else 0.0 for x in shapes]}
    m = normal().mul_(size).mul_(0.3 * used * zero)
    v = normal().square_().mul_(0.2).add_(0.1).mul_(size).mul_(size).mul_(used * zero)
    if case["bits"] == 32:
        s["M"], s["V"] = m, v
    else:
        s["M"], s["ms"] = _encode(m, torch.full_like(m, 0.5), 0.0)
        s["V"], s["vs"] = _encode(v.sqrt_(), torch.full_like(v, 0.5), 1.0)
        # per tensor: its blocks' scales of m, then those of s
        nb = [r // BLOCK for r in room]
        s["S"] = torch.cat([torch.cat((s["ms"][a // BLOCK:a // BLOCK + b], s["vs"][a // BLOCK:a // BLOCK + b]))
                            for a, b in zip(starts, nb)]).view(torch.float8_e8m0fnu)
        at = torch.tensor([[a // BLOCK, b] for a, b in zip(starts, nb)], device="cuda")
        base = torch.repeat_interleave(at[:, 0], at[:, 1])
        s["mi"] = base + torch.arange(total // BLOCK, device="cuda")   # where a block's scale of m stands
        s["vi"] = s["mi"] + torch.repeat_interleave(at[:, 1], at[:, 1])
        s["first"] = torch.repeat_interleave(base * BLOCK, BLOCK)      # start of an element's tensor
        del s["ms"], s["vs"]
    s["list"] = [_views(s, *a) for a in zip(shapes, sizes, starts)]
    return s


def _views(s, shape, n, at):
    parts = [s[k][at:at + n].view(shape) for k in ("X", "G", "M", "V")]
    if s["case"]["bits"] == 8:
        nb = -(-n // BLOCK)
        parts.append(s["S"][2 * at // BLOCK:2 * at // BLOCK + 2 * nb])
    return tuple(parts)


def _adamw_outputs(s):
    return {k: s[k] for k in ("X", "M", "V", "S") if k in s}


# --- plain forms (float32) ------------------------------------------------------

def _update(s, m, root):
    """X from the new first moment and the root of the second."""
    x, d = s["X"], s["decayed"]
    x[:d].mul_(1.0 - LR * DECAY)
    x.sub_(m / (root * (1.0 - BETA2 ** STEP) ** -0.5 + EPS) * (LR / (1.0 - BETA1 ** STEP)))


def _adamw_plain(s):
    g = s["G"].float() * s["scale"]
    m, v = s["M"], s["V"]
    m.mul_(BETA1).add_(g * (1.0 - BETA1))
    v.mul_(BETA2).add_(g * g * (1.0 - BETA2))
    _update(s, m, v.sqrt())
    return _adamw_outputs(s)


def _power(e):
    """2^(e - 127), for the bytes e of normal numbers, or 2^-127 for e = 0."""
    return torch.where(e > 0, e << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _encode(x, u, least):
    """Codes and block scales of x with the dither u; `least`: of a nonzero
    value's code, in ulps."""
    a = x.abs().view(-1, BLOCK)
    byte = ((a.amax(1).view(torch.int32) >> 23) - 7).clamp(min=1)
    a = (a * _power(254 - byte)[:, None]).view(-1)
    e = ((a.view(torch.int32) >> 23) - 127).clamp(min=-6)
    q = (a * _power(130 - e) + u).floor().clamp(min=least)
    code = torch.where(a > 0, q * _power(e + 124), 0.0)
    return torch.where(x < 0, -code, code).to(torch.float8_e4m3fn), byte.to(torch.uint8)


def _dither(s):
    i = torch.arange(s["X"].numel(), device="cuda") - s["first"]
    h = (i + SEED * 0x632BE5AB) * 0x9E3779B1 & 0xffffffff
    h = (h ^ (h >> 15)) * 0x85EBCA77 & 0xffffffff
    h = h ^ (h >> 13)
    return (h & 0xffff).float() * 2.0 ** -16, (h >> 16).float() * 2.0 ** -16


def _adamw8_plain(s):
    scale = _power(s["S"].view(torch.uint8).to(torch.int32))
    m = (s["M"].float().view(-1, BLOCK) * scale[s["mi"]][:, None]).view(-1)
    root = (s["V"].float().view(-1, BLOCK) * scale[s["vi"]][:, None]).view(-1)
    g = s["G"].float() * s["scale"]
    m = m * BETA1 + g * (1.0 - BETA1)
    root = (root * root * BETA2 + g * g * (1.0 - BETA2)).sqrt()
    _update(s, m, root)
    um, uv = _dither(s)
    mc, mb = _encode(m, um, 0.0)
    vc, vb = _encode(root, uv, 1.0)
    s["M"].copy_(mc)
    s["V"].copy_(vc)
    out = s["S"].view(torch.uint8)
    out[s["mi"]] = mb
    out[s["vi"]] = vb
    return _adamw_outputs(s)


def _logits(s):
    return s["x"].float() @ s["w"].float().t()


def _forward_plain(s, case):
    z, y, e = _logits(s), s["y"], case["smoothing"]
    top = z.amax(1)
    rest = (z - top[:, None]).exp().sum(1).log()
    lse = top + rest
    hit = z.gather(1, y.clamp(min=0)[:, None])[:, 0]
    loss = rest + (1.0 - e) * (top - hit) + case["z_loss"] * lse * lse
    if e:
        loss = loss + e * (top - z.mean(1))
    s["loss"].copy_(torch.where(y != IGNORE, loss, 0.0))
    s["lse"].copy_(lse)
    return {"loss": s["loss"], "lse": s["lse"]}


def _backward_plain(s, case):
    y, e, lse = s["y"], case["smoothing"], s["lse"]
    c = torch.where(y != IGNORE, s["dloss"], 0.0)
    dz = (_logits(s) - lse[:, None]).exp() * (c * (1.0 + 2.0 * case["z_loss"] * lse))[:, None]
    if e:
        dz = dz - (c * (e / case["n"]))[:, None]
    dz.scatter_add_(1, y.clamp(min=0)[:, None], (c * (e - 1.0))[:, None])
    s["dx"].copy_(dz @ s["w"].float())
    s["dw"].copy_(dz.t() @ s["x"].float())
    return {"dx": s["dx"], "dw": s["dw"]}


# --- definitions in float64 ----------------------------------------------------

def _adamw64(s, case):
    x, g = s["X"].double(), s["G"].double() * float(s["scale"])
    pad = [torch.full((r,), w, dtype=torch.float64, device="cuda") for w, r in zip(s["wd"], s["room"])]
    if case["bits"] == 32:
        m, v = s["M"].double(), s["V"].double()
    else:
        unit = torch.exp2(s["S"].view(torch.uint8).double() - 127.0)
        m = s["M"].double() * unit[s["mi"]].repeat_interleave(BLOCK)
        v = (s["V"].double() * unit[s["vi"]].repeat_interleave(BLOCK)).square()
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g.square()
    hat = m / (1.0 - BETA1 ** STEP)
    x = x - LR * torch.cat(pad) * x - LR * hat / ((v / (1.0 - BETA2 ** STEP)).sqrt() + EPS)
    if case["bits"] == 32:
        return {"X": x, "M": m, "V": v}
    number = torch.cat([torch.arange(r, device="cuda") for r in s["room"]])
    number = ((number + SEED * 0x632BE5AB) % 2 ** 32) * 0x9E3779B1 % 2 ** 32
    number = torch.bitwise_xor(number, number // 2 ** 15) * 0x85EBCA77 % 2 ** 32
    number = torch.bitwise_xor(number, number // 2 ** 13)
    mv, me = _round64(m, (number % 2 ** 16).double() / 2 ** 16, False)
    rv, re = _round64(v.sqrt(), (number // 2 ** 16).double() / 2 ** 16, True)
    at = torch.empty(2 * len(me), dtype=torch.float64, device="cuda")
    at[s["mi"]], at[s["vi"]] = torch.exp2(me), torch.exp2(re)
    return {"X": x, "M": mv, "V": rv, "S": at}


def _round64(x, u, nonzero):
    """e4m3 values of x over its blocks' powers of two, and their exponents."""
    a = x.abs().reshape(-1, BLOCK)
    top = a.amax(1)
    exponent = (torch.frexp(top)[1].double() - 8.0).clamp(min=-126.0)
    exponent = torch.where(top > 0, exponent, -126.0)
    a = a * torch.exp2(-exponent)[:, None]
    ulp = torch.exp2((torch.frexp(a)[1].double() - 1.0).clamp(min=-6.0) - 3.0)
    q = torch.floor(a / ulp + u.reshape(-1, BLOCK))
    if nonzero:
        q = q.clamp(min=1.0)
    return (torch.sign(x).reshape(-1, BLOCK) * q * ulp).reshape(-1), exponent
