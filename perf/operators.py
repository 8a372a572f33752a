"""What the Muon operators are measured on: muon_orthogonalize (the
Newton-Schulz orthogonalisation of a matrix or a batch of them) and muon_step
(momentum kept in fp32, bf16 or 8 bits, orthogonalised and applied to fp32
params), each over the range from a few small matrices to a large model's
largest ones.

With `own` false, run() computes the plain forms: elementary torch operations
in 32 bits (the 8-bit codes' borders in the rounding order the format
defines).  With `own` true it makes the library's calls.
"""
import math

import torch

own = False

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
BLOCK = 2048
TINY = 2.0 ** -112


# --------------------------------------------------------------------- cases
def _orth(name, batch, rows, cols, dtype):
    return {"name": name, "op": "orthogonalize", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype}


def _step(name, shapes, storage, grads, **more):
    case = {"name": name, "op": "step", "shapes": shapes, "storage": storage, "grads": grads, "stochastic": False,
            "nesterov": True, "scale": "rms"}
    case.update(more)
    return case


def listed():
    return [
        # one small matrix (an adapter's factor): the time is latency alone
        _orth("orth_one_small", 1, 48, 80, "f32"),
        # attention projections split by head, each head on its own
        _orth("orth_heads", 96, 64, 768, "bf16"),
        # one classifier head: a long side that is no multiple of a tile
        _orth("orth_head_ragged", 1, 1000, 768, "f32"),
        # the fused query-key-value weights of twelve encoder blocks, tall
        _orth("orth_qkv_12", 12, 2304, 768, "bf16"),
        # a wide square projection
        _orth("orth_square", 1, 2048, 2048, "f32"),
        # a large model's up projection, gradient in bf16
        _orth("orth_mlp_large", 1, 11008, 4096, "bf16"),
        # a few small odd matrices: a step that is all latency
        _step("step_small_odd", "33x65,128x64,1x77,200x31,64x64", "f32", "f32", scale="spectral"),
        # the attention weights of twelve encoder blocks, momentum in bf16
        _step("step_encoder_attention", ",".join(["2304x768,768x768"] * 12), "bf16", "f32"),
        # the same in 8 bits, nearest rounding, without Nesterov
        _step("step_encoder_attention_q8", ",".join(["2304x768,768x768"] * 12), "q8", "f32", nesterov=False),
        # one decoder layer, bf16 gradients, 8-bit momentum rounded stochastically
        _step("step_decoder_layer_q8_sr", "2048x6144,2048x2048,2048x8192,8192x2048", "q8", "bf16", stochastic=True),
        # a large layer's four attention projections, fp32 momentum
        _step("step_projections_large", "4096x4096,4096x4096,4096x4096,4096x4096", "f32", "bf16"),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _flops(rows, cols):
    m, n = min(rows, cols), max(rows, cols)
    # X X^T and A^2 are symmetric (half of a product each), B X is whole
    return STEPS * (float(m) * m * n + float(m) * m * m + 2.0 * m * m * n)


def draw(rng):
    if rng.random() < 0.5:
        while True:
            rows, cols = _log_int(rng, 16, 6000), _log_int(rng, 16, 6000)
            batch = _log_int(rng, 1, 48)
            if batch * _flops(rows, cols) <= 1.2e12 and batch * rows * cols <= 6e7:
                break
        case = _orth("", batch, rows, cols, rng.choice(["f32", "bf16"]))
    else:
        while True:
            shapes = []
            for _ in range(rng.randint(1, 4)):
                one = (_log_int(rng, 24, 4500), _log_int(rng, 24, 4500))
                shapes += [one] * rng.randint(1, 5)
            if sum(_flops(*s) for s in shapes) <= 1.0e12 and sum(a * b for a, b in shapes) <= 5e7:
                break
        storage = rng.choice(["f32", "bf16", "q8"])
        case = _step("", ",".join("%dx%d" % s for s in shapes), storage, rng.choice(["f32", "bf16"]),
                     stochastic=storage == "q8" and rng.random() < 0.5, nesterov=rng.random() < 0.7,
                     scale=rng.choice(["rms", "spectral", "none"]))
    del case["name"]
    return case


def _shapes(case):
    return [tuple(int(x) for x in s.split("x")) for s in case["shapes"].split(",")]


def work(case):
    if case["op"] == "orthogonalize":
        n = case["batch"] * case["rows"] * case["cols"]
        return {"bytes": n * (8 if case["dtype"] == "f32" else 4),
                "flops": case["batch"] * _flops(case["rows"], case["cols"])}
    shapes = _shapes(case)
    n = sum(a * b for a, b in shapes)
    blocks = sum(-(-a * b // BLOCK) for a, b in shapes)
    # params and momentum read and written, grads read, and the momentum's
    # values written as they are handed back (bf16, or fp32)
    per = 8 + (4 if case["grads"] == "f32" else 2) + {"f32": 8 + 4, "bf16": 4 + 2, "q8": 2 + 4}[case["storage"]]
    return {"bytes": n * per + (8 * blocks if case["storage"] == "q8" else 0),
            "flops": sum(_flops(*z) for z in shapes)}


# -------------------------------------------------------------------- inputs
def _gradient(gen, shape, size):
    """A gradient-like matrix: a few directions that matter over noise."""
    rows, cols = shape[-2:]
    rank = max(1, min(rows, cols) // 16)
    left = torch.randn(*shape[:-2], rows, rank, generator=gen, device="cuda")
    right = torch.randn(*shape[:-2], rank, cols, generator=gen, device="cuda")
    noise = torch.randn(*shape, generator=gen, device="cuda")
    return (left @ right).mul_(1.0 / math.sqrt(rank)).add_(noise, alpha=0.1).mul_(size)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] == "orthogonalize":
        x = _gradient(gen, (case["batch"], case["rows"], case["cols"]), 1e-3)
        return {"case": case, "x": x if case["dtype"] == "f32" else x.to(torch.bfloat16)}
    shapes = _shapes(case)
    s = {"case": case, "shapes": shapes, "t": 11, "seed": 1000 + int(seed) % 1000,
         "hp": {"lr": 2e-3, "momentum": 0.95, "weight_decay": 0.01}}
    s["params"] = [torch.randn(*z, generator=gen, device="cuda").mul_(0.02) for z in shapes]
    grads = [_gradient(gen, z, 1e-3) for z in shapes]
    s["grads"] = grads if case["grads"] == "f32" else [g.to(torch.bfloat16) for g in grads]
    # the momentum of earlier steps, in its storage
    s["stored"] = [_encode(_gradient(gen, z, 4e-4), case["storage"]) for z in shapes]
    if own:
        import memory_efficient_adam_amd as ma
        s["state"] = ma.muon_state_create(shapes, case["storage"], case["grads"])
        _fill(ma, s["state"], s.pop("stored"), shapes, case["storage"])
    return s


def _fill(ma, state, stored, shapes, storage):
    """The momentum of `stored` into a library state's buffers (each matrix's
    segment padded to 16 entries)."""
    name = {"f32": "m_f32", "bf16": "m_bf16", "q8": "m_codes"}[storage]
    parts = []
    for v, z in zip(stored, shapes):
        flat = (v[0] if storage == "q8" else v).reshape(-1)
        parts += [flat, flat.new_zeros(-flat.numel() % 16)]
    ma.muon_state_write(state, name, torch.cat(parts))
    if storage == "q8":
        ma.muon_state_write(state, "m_scale", torch.cat([v[1] for v in stored]))


# --------------------------------------------------------------- plain forms
def _plain_orthogonalize(u):
    """fp32 throughout; u is (..., rows, cols)."""
    tall = u.shape[-2] > u.shape[-1]
    x = u.float()
    if tall:
        x = x.transpose(-2, -1).contiguous()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = x @ x.transpose(-2, -1)
        poly = b * gram + c * (gram @ gram)
        x = a * x + poly @ x
    return x.transpose(-2, -1).contiguous() if tall else x


def _blocks(flat):
    short = -flat.numel() % BLOCK
    return torch.nn.functional.pad(flat, (0, short)).view(-1, BLOCK)


def _philox_low16(first, count, t, seed):
    """The 16-bit draws of `count` elements from draw index `first` (a multiple
    of 16): Philox4x32-10 at counter (index / 4, t), word index mod 4, low half."""
    mask = 0xFFFFFFFF
    groups = first // 4 + torch.arange(-(-count // 4), device="cuda", dtype=torch.int64)
    c0, c1 = groups & mask, groups >> 32
    c2, c3 = torch.full_like(c0, t & mask), torch.full_like(c0, t >> 32)
    k0, k1 = seed & mask, seed >> 32

    def product(k, c):  # 32 x 32 -> 64 bits, as (high, low)
        low, high = k * (c & 0xFFFF), k * (c >> 16)
        return (high + (low >> 16)) >> 16, (((high & 0xFFFF) << 16) + low) & mask

    for _ in range(10):
        h0, l0 = product(0xD2511F53, c0)
        h1, l1 = product(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    return (torch.stack((c0, c1, c2, c3), 1).reshape(-1) & 0xFFFF)[:count]


def _encode(m, storage, draws=None):
    """fp32 momentum in its storage: itself, bf16, or (int8 codes, fp32 block scales)."""
    if storage == "f32":
        return m
    if storage == "bf16":
        return m.to(torch.bfloat16)
    x = _blocks(m.reshape(-1))
    scale = x.abs().amax(1, keepdim=True)
    live = scale >= TINY
    y = x.abs() * (127.0 / torch.where(live, scale, 1.0))
    if draws is None:
        k = y.round()
    else:
        down = y.floor()
        k = down + (_blocks(draws.float()) * 2.0 ** -16 < y - down)
    k = torch.where(x.abs() >= scale, 127.0, k.clamp(max=127.0))
    k = torch.where(live, k.copysign(x), 0.0)
    return (k.reshape(-1)[:m.numel()].to(torch.int8).view(m.shape), torch.where(live, scale, 0.0).reshape(-1))


def _decode(stored, storage):
    if storage != "q8":
        return stored.float()
    codes, scale = stored
    x = _blocks(codes.reshape(-1).float()) * torch.tensor(1.0 / 127.0, device=codes.device) * scale[:, None]
    return x.reshape(-1)[:codes.numel()].view(codes.shape)


def _fma(a, x, y):
    """a * x + y rounded once to fp32 (the product is exact in 64 bits)."""
    return (x.double() * a + y.double()).float()


def _f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def _factor(shape, scale):
    rows, cols = shape
    return {"none": 1.0, "spectral": math.sqrt(max(1.0, rows / cols)), "rms": 0.2 * math.sqrt(max(rows, cols))}[scale]


def _plain_step(s):
    case, hp = s["case"], s["hp"]
    storage = case["storage"]
    beta = _f32(hp["momentum"])
    rest = _f32(1.0 - beta)
    lr, decay = _f32(hp["lr"]), _f32(1.0 - _f32(hp["lr"]) * _f32(hp["weight_decay"]))
    new, updates, first = [], [], 0
    for g, stored in zip(s["grads"], s["stored"]):
        part = g.float() * rest
        m = _fma(beta, _decode(stored, storage), part)
        draws = _philox_low16(first, m.numel(), s["t"], s["seed"]) if case["stochastic"] else None
        new.append(_encode(m, storage, draws))
        updates.append(_fma(beta, m, part) if case["nesterov"] else m)
        first += -(-m.numel() // 16) * 16
    # matrices of one shape go through the products together
    for shape in dict.fromkeys(s["shapes"]):
        at = [k for k, z in enumerate(s["shapes"]) if z == shape]
        o = _plain_orthogonalize(torch.stack([updates[k] for k in at]))
        rate = _f32(lr * _factor(shape, case["scale"]))
        for k, one in zip(at, o):
            s["params"][k].mul_(decay).sub_(one, alpha=rate)
    s["stored"] = new
    s["t"] += 1
    return {"params": s["params"], "momentum": [_decode(v, "q8") if storage == "q8" else v for v in new]}


# ----------------------------------------------------------------------- run
def run(state):
    case = state["case"]
    if case["op"] == "orthogonalize":
        if own:
            import memory_efficient_adam_amd as ma
            return ma.muon_orthogonalize(state["x"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        return _plain_orthogonalize(state["x"]).to(state["x"].dtype)
    if own:
        import memory_efficient_adam_amd as ma
        ma.muon_step(state["state"], state["params"], state["grads"], t=state["t"], nesterov=case["nesterov"],
                     steps=STEPS, coefficients=COEFFICIENTS, eps=EPS, scale=case["scale"],
                     stochastic=case["stochastic"], seed=state["seed"], **state["hp"])
        state["t"] += 1
        return {"params": state["params"], "momentum": ma.muon_state_momentum(state["state"])}
    return _plain_step(state)


# --------------------------------------------------------------------- exact
def _exact_orthogonalize(u):
    """The same polynomial in 64 bits, through the short side's Gram matrix:
    X_K = P_K .. P_1 X_0 with P = a I + b A + c A^2 and A <- P A P."""
    x = u.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + EPS)
    gram = x.mT.contiguous() @ x if tall else x @ x.mT.contiguous()
    a, b, c = COEFFICIENTS
    eye = torch.eye(gram.shape[-1], dtype=torch.float64, device=x.device)
    whole = None
    for _ in range(STEPS):
        p = a * eye + gram @ (b * eye + c * gram)
        whole = p if whole is None else p @ whole
        gram = p @ gram @ p
    return x @ whole if tall else whole @ x


def exact(case, seed):
    state = prepare(case, seed) if not own else None
    if case["op"] == "orthogonalize":
        return torch.stack([_exact_orthogonalize(x) for x in state["x"]])
    beta, lr, wd = (_f32(state["hp"][k]) for k in ("momentum", "lr", "weight_decay"))
    params, momentum = [], []
    for p, g, stored, shape in zip(state["params"], state["grads"], state["stored"], state["shapes"]):
        if case["storage"] == "q8":  # what the codes stand for: code / 127 of the block's scale
            old = _blocks(stored[0].reshape(-1).double()) / 127.0 * stored[1].double()[:, None]
            old = old.reshape(-1)[:p.numel()].view(shape)
        else:
            old = stored.double()
        m = beta * old + (1.0 - beta) * g.double()
        u = beta * m + (1.0 - beta) * g.double() if case["nesterov"] else m
        params.append(p.double() * (1.0 - lr * wd) - lr * _factor(shape, case["scale"]) * _exact_orthogonalize(u))
        # new 8-bit codes have no value apart from fp32's rounding order, which defines them
        momentum.append(None if case["storage"] == "q8" else m)
    return {"params": params, "momentum": momentum}
