"""What the embedding operators and the step with 32-bit states are measured
on: adam_step_noalloc with both moments in fp32, embedding_lookup (rows of a
table by token, scaled), embedding_gradient (its gradient, dense, written or
added) and embedding_adam_step (the fp32-state step on the rows that tokens
name), each over the range from a few rows to a large model's batch.

With `own` false, run() computes the plain forms: elementary torch operations
in 32 bits.  With `own` true it makes the library's calls.
"""
import functools
import math

import torch

own = False

HP = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01}
FIRST_STEP = 11


# --------------------------------------------------------------------- cases
def _adam(name, sizes, grads, amsgrad=False, decoupled=True):
    return {"name": name, "op": "adam", "sizes": sizes, "grads": grads, "amsgrad": amsgrad, "decoupled": decoupled}


def _lookup(name, tokens, rows, cols, table, out, ids, scale):
    return {"name": name, "op": "lookup", "tokens": tokens, "rows": rows, "cols": cols, "table": table, "out": out,
            "ids": ids, "scale": scale, "padding": 0.0}


def _gradient(name, tokens, rows, cols, grads, out, ids, scale, accumulate=False, padding=0.0):
    return {"name": name, "op": "gradient", "tokens": tokens, "rows": rows, "cols": cols, "grads": grads, "out": out,
            "ids": ids, "scale": scale, "accumulate": accumulate, "padding": padding}


def _rows(name, tokens, rows, cols, grads, ids, scale, amsgrad=False, decoupled=True, padding=0.0):
    return {"name": name, "op": "rows", "tokens": tokens, "rows": rows, "cols": cols, "grads": grads, "ids": ids,
            "scale": scale, "amsgrad": amsgrad, "decoupled": decoupled, "padding": padding}


_BLOCK_2048 = "2048,2048,12582912,6144,4194304,2048,2048,2048,16777216,8192,16777216,2048"


def listed():
    return [
        # sixteen small ragged tensors (norms, biases, adapters): launch and host time
        _adam("adam_small_ragged", "1,3,4,5,16,17,1000,1023,1024,1025,2047,2048,2049,4096,6001,12289", "f32"),
        # three decoder blocks of width 2048, 36 tensors, fp32 gradients
        _adam("adam_three_blocks", ",".join([_BLOCK_2048] * 3), "f32"),
        # a token and a position table with AMSGrad, bf16 gradients
        _adam("adam_tables_amsgrad", "103022592,4194304", "bf16", amsgrad=True),
        # serving: one token for each of eight sequences, bf16 table
        _lookup("lookup_decode", 8, 32000, 4096, "bf16", "bf16", "i64", 1.0),
        # a training batch of 8 x 2048 tokens, bf16 activations straight from the fp32 table
        _lookup("lookup_batch", 16384, 50304, 2048, "f32", "bf16", "i64", math.sqrt(2048.0)),
        # an odd width, as a table of features has, in fp32 throughout
        _lookup("lookup_odd", 20011, 32000, 771, "f32", "f32", "i32", 1.0),
        # a short batch into a small table of odd width, everything of it latency
        _gradient("gradient_small", 333, 1000, 771, "f32", "f32", "i32", 1.0),
        # the dense gradient of a training batch of 8 x 2048 tokens
        _gradient("gradient_batch", 16384, 50304, 2048, "bf16", "f32", "i64", math.sqrt(2048.0)),
        # 32 x 2048 tokens, a tenth of them padding, added to the gradient that a tied head left
        _gradient("gradient_tied_large", 65536, 32000, 4096, "bf16", "f32", "i64", 1.0, accumulate=True, padding=0.1),
        # a short batch's rows of a table, stepped at once
        _rows("rows_small", 500, 32000, 770, "f32", "i32", 1.0, decoupled=False),
        # the rows of a training batch of 8 x 2048 tokens
        _rows("rows_batch", 16384, 50304, 2048, "bf16", "i64", math.sqrt(2048.0)),
        # the rows of a large batch with AMSGrad, a tenth of the tokens padding
        _rows("rows_large", 65536, 32000, 4096, "bf16", "i64", 1.0, amsgrad=True, padding=0.1),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["adam", "lookup", "gradient", "rows"])
    types = ["f32", "bf16"]
    if op == "adam":
        while True:
            sizes = []
            for _ in range(rng.randint(1, 4)):
                sizes += [_log_int(rng, 1, 6e7)] * rng.randint(1, 8)
            if sum(sizes) <= 1.3e8:
                break
        case = _adam("", ",".join(map(str, sizes)), rng.choice(types), rng.random() < 0.3, rng.random() < 0.7)
    else:
        while True:
            tokens, rows, cols = _log_int(rng, 1, 65536), _log_int(rng, 16, 130000), _log_int(rng, 16, 4096)
            if rng.random() < 0.6:  # most widths are multiples of 64, some are odd
                cols = max(64, cols // 64 * 64)
            if tokens * cols <= 2.0e8 and rows * cols <= 1.1e8:
                break
        ids, scale = rng.choice(["i32", "i64"]), rng.choice([1.0, math.sqrt(cols)])
        padding = rng.choice([0.0, 0.0, 0.1, 0.4])
        if op == "lookup":
            case = _lookup("", tokens, rows, cols, rng.choice(types), rng.choice(types), ids, scale)
            case["padding"] = padding
        elif op == "gradient":
            case = _gradient("", tokens, rows, cols, rng.choice(types), rng.choice(types), ids, scale,
                             rng.random() < 0.4, padding)
        else:
            case = _rows("", tokens, rows, cols, rng.choice(types), ids, scale, rng.random() < 0.3,
                         rng.random() < 0.7, padding)
    del case["name"]
    return case


def _sizes(case):
    return [int(n) for n in case["sizes"].split(",")]


@functools.lru_cache(maxsize=64)
def _different(tokens, rows):
    """Expected number of different rows among `tokens` draws of _tokens."""
    k = torch.arange(1, rows + 1, dtype=torch.float64)
    p = torch.log1p(1.0 / k) / math.log(rows + 1.0)
    return float((1.0 - torch.exp(tokens * torch.log1p(-p))).sum())


_BYTES = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}


def work(case):
    if case["op"] == "adam":
        n = sum(_sizes(case))
        per = 24 + _BYTES[case["grads"]] + (8 if case["amsgrad"] else 0)
        return {"bytes": n * per, "flops": n * 16}
    inside = case["tokens"] * (1.0 - case["padding"])
    cols, rows = case["cols"], case["rows"]
    ids, different = case["tokens"] * _BYTES[case["ids"]], _different(round(inside), rows)
    if case["op"] == "lookup":
        return {"bytes": int(ids + different * cols * _BYTES[case["table"]] + case["tokens"] * cols * _BYTES[case["out"]]),
                "flops": int(inside * cols)}
    taken = ids + inside * cols * _BYTES[case["grads"]]
    if case["op"] == "gradient":
        put = 2 * different * cols if case["accumulate"] else rows * cols
        return {"bytes": int(taken + put * _BYTES[case["out"]]), "flops": int(inside * cols + different * cols)}
    per = 24 + (8 if case["amsgrad"] else 0)
    return {"bytes": int(taken + different * cols * per), "flops": int(inside * cols + 17 * different * cols)}


# -------------------------------------------------------------------- inputs
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32, "i64": torch.int64}


def _tokens(gen, case):
    """Tokens by rank-frequency (the k-th most frequent row's share falls as 1/k,
    as words do), the ranks spread over the table; padding is -1."""
    rows, n = case["rows"], case["tokens"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(rows + 1.0)) - 1.0).long().clamp_(0, rows - 1)
    tokens = torch.randperm(rows, generator=gen, device="cuda")[rank]
    if case["padding"] > 0.0:
        absent = torch.rand(n, generator=gen, device="cuda") < case["padding"]
        tokens = torch.where(absent, -1, tokens)
    return tokens.to(_TYPES[case["ids"]])


def _normal(gen, shape, size, dtype="f32"):
    return torch.randn(shape, generator=gen, device="cuda").mul_(size).to(_TYPES[dtype])


def _state(gen, sizes, amsgrad):
    """Moments of earlier steps in the layout of caller-owned buffers: each
    tensor's segment padded to 16 entries; and the tensors' own views of them."""
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // 16) * 16
    flat = {"m_f32": _normal(gen, total, 1e-4), "v_f32": _normal(gen, total, 1e-3).square_()}
    for b in flat.values():
        for s, n in zip(starts, sizes):
            b[s + n:s + n + -n % 16] = 0.0
    if amsgrad:
        flat["vmax_f32"] = flat["v_f32"] * (1.0 + 0.5 * torch.rand(total, generator=gen, device="cuda"))
    views = {k: [b[s:s + n] for s, n in zip(starts, sizes)] for k, b in flat.items()}
    return flat, views


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case, "t": FIRST_STEP}
    if case["op"] == "adam":
        sizes = _sizes(case)
        s["params"] = [_normal(gen, n, 0.02) for n in sizes]
        s["grads"] = [_normal(gen, n, 1e-3, case["grads"]) for n in sizes]
        s["buffers"], s["views"] = _state(gen, sizes, case["amsgrad"])
        return s
    s["tokens"] = _tokens(gen, case)
    shape = (case["rows"], case["cols"])
    if case["op"] == "lookup":
        s["table"] = _normal(gen, shape, 0.02, case["table"])
        return s
    s["grad"] = _normal(gen, (case["tokens"], case["cols"]), 1e-3, case["grads"])
    if case["op"] == "gradient":
        if case["accumulate"]:
            s["sum"] = _normal(gen, shape, 1e-2, case["out"])
    else:
        s["table"] = _normal(gen, shape, 0.02)
        s["buffers"], s["views"] = _state(gen, [shape[0] * shape[1]], case["amsgrad"])
    if own:
        import memory_efficient_adam_amd as ma
        need = ma.embedding_gradient_workspace_bytes(case["tokens"], *shape)
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------- plain forms
def _f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def _scalars(t):
    """The hyperparameters as fp32 holds them, and what follows from them in 64 bits."""
    h = {k: _f32(v) for k, v in HP.items()}
    return {**h, "rate": h["lr"] / (1.0 - h["beta1"] ** t), "root": 1.0 / math.sqrt(1.0 - h["beta2"] ** t),
            "decay": 1.0 - h["lr"] * h["weight_decay"]}


def _update(p, g, m, v, w, h, decoupled):
    """One step on fp32 tensors, in place."""
    if not decoupled:
        g = g.add(p, alpha=h["weight_decay"])
    m.mul_(h["beta1"]).add_(g, alpha=1.0 - h["beta1"])
    v.mul_(h["beta2"]).addcmul_(g, g, value=1.0 - h["beta2"])
    if w is not None:
        torch.maximum(w, v, out=w)
    below = (v if w is None else w).sqrt().mul_(h["root"]).add_(h["eps"])
    if decoupled:
        p.mul_(h["decay"])
    p.addcdiv_(m, below, value=-h["rate"])


def _plain_adam(s):
    h, views = _scalars(s["t"]), s["views"]
    for k, (p, g) in enumerate(zip(s["params"], s["grads"])):
        w = views["vmax_f32"][k] if s["case"]["amsgrad"] else None
        _update(p, g.float(), views["m_f32"][k], views["v_f32"][k], w, h, s["case"]["decoupled"])


def _plain_lookup(s):
    case, tokens = s["case"], s["tokens"].long()
    x = s["table"][tokens.clamp(min=0)].float()
    if case["scale"] != 1.0:
        x = x.mul_(case["scale"])
    if case["padding"] > 0.0:
        x = torch.where((tokens < 0)[:, None], 0.0, x)
    return x.to(_TYPES[case["out"]])


def _plain_gradient(s):
    case, tokens, grad = s["case"], s["tokens"].long(), s["grad"].float()
    if case["padding"] > 0.0:
        grad = torch.where((tokens < 0)[:, None], 0.0, grad)
        tokens = tokens.clamp(min=0)
    if case["accumulate"] and case["out"] == "f32":
        return s["sum"].index_add_(0, tokens, grad, alpha=case["scale"])
    total = torch.zeros(case["rows"], case["cols"], device="cuda").index_add_(0, tokens, grad, alpha=case["scale"])
    if case["accumulate"]:
        return s["sum"].copy_(total.add_(s["sum"]))
    return total.to(_TYPES[case["out"]])


def _plain_rows(s):
    case, tokens, grad, h = s["case"], s["tokens"].long(), s["grad"].float(), _scalars(s["t"])
    if case["padding"] > 0.0:
        inside = tokens >= 0
        tokens, grad = tokens[inside], grad[inside]
    named, back = torch.unique(tokens, return_inverse=True)
    g = torch.zeros(named.numel(), case["cols"], device="cuda").index_add_(0, back, grad, alpha=case["scale"])
    names = ["m_f32", "v_f32"] + (["vmax_f32"] if case["amsgrad"] else [])
    whole = [s["table"]] + [s["views"][k][0].view_as(s["table"]) for k in names]
    part = [x[named] for x in whole]
    _update(part[0], g, part[1], part[2], part[3] if case["amsgrad"] else None, h, case["decoupled"])
    for x, y in zip(whole, part):
        x[named] = y


# ----------------------------------------------------------------------- run
def _stepped(s):
    params = s["params"] if s["case"]["op"] == "adam" else [s["table"]]
    return {"params": params, **s["buffers"]}


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "lookup":
            return _plain_lookup(state)
        if case["op"] == "gradient":
            return _plain_gradient(state)
        (_plain_adam if case["op"] == "adam" else _plain_rows)(state)
        state["t"] += 1
        return _stepped(state)
    import memory_efficient_adam_amd as ma
    if case["op"] == "adam":
        ma.adam_step_noalloc(state["params"], state["grads"], state["buffers"], storage="f32", grad_dtype=case["grads"],
                             amsgrad=case["amsgrad"], decoupled=case["decoupled"], t=state["t"], **HP)
    elif case["op"] == "lookup":
        return ma.embedding_lookup(state["table"], state["tokens"], scale=case["scale"], dtype=_TYPES[case["out"]])
    elif case["op"] == "gradient":
        return ma.embedding_gradient(state["grad"], state["tokens"], case["rows"], scale=case["scale"],
                                     dtype=_TYPES[case["out"]], out=state.get("sum"), accumulate=case["accumulate"],
                                     workspace=state["workspace"])
    else:
        ma.embedding_adam_step(state["table"], state["grad"], state["tokens"], state["buffers"],
                               amsgrad=case["amsgrad"], decoupled=case["decoupled"], scale=case["scale"],
                               t=state["t"], workspace=state["workspace"], **HP)
    state["t"] += 1
    return _stepped(state)


# --------------------------------------------------------------------- exact
def _exact_update(p, g, m, v, w, h, decoupled):
    p = p.double()
    g = g if decoupled else g + h["weight_decay"] * p
    m = h["beta1"] * m.double() + (1.0 - h["beta1"]) * g
    v = h["beta2"] * v.double() + (1.0 - h["beta2"]) * g * g
    w = None if w is None else torch.maximum(w.double(), v)
    top = p * (1.0 - h["lr"] * h["weight_decay"]) if decoupled else p
    p = top - h["rate"] * m / ((v if w is None else w).sqrt() * h["root"] + h["eps"])
    return [p, m, v] + ([] if w is None else [w])


def _joined(flat, parts):
    """The tensors' values in the buffer's layout (segments padded with zeros to 16 entries)."""
    padded = [torch.nn.functional.pad(x.reshape(-1), (0, -x.numel() % 16)) for x in parts]
    return torch.cat(padded).view_as(flat)


def exact(case, seed):
    s = prepare(case, seed)
    h = _scalars(s["t"])
    names = ["params", "m_f32", "v_f32"] + (["vmax_f32"] if case.get("amsgrad") else [])
    if case["op"] == "adam":
        new = [_exact_update(p, g.double(), *(s["views"][k][i] for k in names[1:]),
                             *([] if case["amsgrad"] else [None]), h, case["decoupled"])
               for i, (p, g) in enumerate(zip(s["params"], s["grads"]))]
        return {k: [one[j] for one in new] if k == "params" else _joined(s["buffers"][k], [one[j] for one in new])
                for j, k in enumerate(names)}
    tokens = s["tokens"].long()
    inside = tokens >= 0
    if case["op"] == "lookup":
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        out[inside] = s["table"].double()[tokens[inside]] * _f32(case["scale"])
        return out
    # sums over the tokens of a row: by order of rows and a running sum's differences would lose
    # bits, so one scatter-add in 64 bits
    total = torch.zeros(case["rows"], case["cols"], dtype=torch.float64, device="cuda")
    total.scatter_add_(0, tokens[inside][:, None].expand(-1, case["cols"]), s["grad"][inside].double())
    total *= _f32(case["scale"])
    if case["op"] == "gradient":
        return total + s["sum"].double() if case["accumulate"] else total
    hit = torch.zeros(case["rows"], dtype=torch.bool, device="cuda")
    hit[tokens[inside]] = True
    old = [s["table"]] + [s["views"][k][0].view_as(s["table"]) for k in names[1:]]
    rows = _exact_update(old[0][hit], total[hit], *(x[hit] for x in old[1:]),
                         *([] if case["amsgrad"] else [None]), h, case["decoupled"])
    out = {}
    for k, x, y in zip(names, old, rows):
        whole = x.double()
        whole[hit] = y
        out[k] = [whole] if k == "params" else _joined(s["buffers"][k], [whole])
    return out
