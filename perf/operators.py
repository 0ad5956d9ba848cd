"""Measured cases of the AdamW step with 8-bit moments, of gradient clipping by
the global norm inside the step, and of the conversion between float32 and
8-bit moments.

An AdamW tensor's two moments are held as one byte an element, in blocks of
256 consecutive elements (row-major).  With t the step count, g the gradient
times the clipping factor, all in float32, each operation rounded by itself:

    m' = b1 m + (1-b1) g              v' = b2 v + ((1-b2) g) g
    w' = w - lr wd w - lr (m' / (1-b1^t)) / (sqrt(v' / (1-b2^t)) + eps)

then m' and v' are rounded to their bytes, up or down at random such that the
mean is the value itself:

  first moment   an e4m3 number times 2^(e-127), one e for each block:
                 e = max(((bits(max |m'|) + 0x1fffff) >> 23) - 8, 9)
  second moment  the float32 whose bits are (code + base) << 20, code 1..255,
                 one base for each block, base = max(((bits(max v') + 0xfffff)
                 >> 20) - 255, 0); code 0 is zero, and a value above zero
                 never gets it.

A byte's value is exact in bfloat16.  The random numbers are a function of
(seed, t, tensor, element): a 32-bit word for each element, whose upper 20
bits serve the first moment and whose lower 20 the second.  Conversion from float32 rounds to nearest, ties to even.

Clipping: norm = sqrt(sum of every gradient's squares) over all tensors of the
step, factor = min(1, max_norm / norm).
"""

import math

import numpy as np
import torch

own = False

BLOCK = 256
LR, BETA1, BETA2, EPS, DECAY = (float(np.float32(x)) for x in (3e-4, 0.9, 0.95, 1e-8, 0.01))
MUON_LR, MUON_MU, MUON_EPS, MUON_DECAY = (float(np.float32(x)) for x in (0.02, 0.95, 1e-7, 0.01))
NS_STEPS = 5
NS_A, NS_B, NS_C = (float(np.float32(x)) for x in (3.4445, -4.7750, 2.0315))
STEPS_TAKEN = 1000        # the step count that a state starts from
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the layer norms' gains and biases of a 12-layer, 768-wide model: latency
        {"name": "step_vectors_bf16", "op": "step", "dtype": "bf16", "shapes": "50*768", "clip": 0.0},
        # its position embedding, trained in float32
        {"name": "step_positions_f32", "op": "step", "dtype": "f32", "shapes": "1024x768", "clip": 0.0},
        # adapters, heads and gains of odd sizes side by side
        {"name": "step_ragged_bf16", "op": "step", "dtype": "bf16",
         "shapes": "1,2,255,257,1000,333x65,50257,127x1025,4099x301", "clip": 0.0},
        # the token embedding (the head is tied to it) of the 768-wide model
        {"name": "step_tokens_f32", "op": "step", "dtype": "f32", "shapes": "50257x768", "clip": 0.0},
        # both embeddings of the 1600-wide, 48-layer model: the largest
        {"name": "step_xl_embeddings_bf16", "op": "step", "dtype": "bf16", "shapes": "50257x1600,1024x1600",
         "clip": 0.0},
        # the vectors again, their gradients clipped
        {"name": "clip_vectors_f32", "op": "step", "dtype": "f32", "shapes": "50*768", "clip": 0.5},
        # every AdamW parameter of the 768-wide model under one norm
        {"name": "clip_model_bf16", "op": "step", "dtype": "bf16", "shapes": "50257x768,1024x768,50*768,12*2304",
         "clip": 1.0},
        # two layers' attention matrices (stepped with Muon) and the AdamW tensors beside them under one norm
        {"name": "clip_matrices_bf16", "op": "step", "dtype": "bf16", "shapes": "1024x768,8*768", "clip": 1.0,
         "matrices": 8, "width": 768},
        # a checkpoint's moments read in and written out: the vectors, odd sizes, the token embedding
        {"name": "convert_vectors", "op": "convert", "dtype": "bf16", "shapes": "50*768"},
        {"name": "convert_ragged", "op": "convert", "dtype": "f32", "shapes": "1,257,333x65,50257,127x1025,4099x301"},
        {"name": "convert_tokens", "op": "convert", "dtype": "bf16", "shapes": "50257x768"},
    ]


def draw(rng):
    dtype = rng.choice(["bf16", "f32"])
    most = 40_000_000 if dtype == "bf16" else 25_000_000
    left = int(math.exp(rng.uniform(math.log(2000), math.log(most))))
    parts = []
    for _ in range(rng.randint(1, 24)):     # tensors of a few sizes, the rest of the budget split between them
        n = max(1, min(left, int(left * rng.uniform(0.05, 0.9))))
        cols = rng.choice([1, 64, 65, 301, 768, 1025, 1600, 2304])
        rows = max(1, n // cols)
        if rng.random() < 0.4 or rows >= 1 << 20:
            parts.append(str(min(rows * cols + rng.randint(0, 7), 1 << 20)))
        else:
            parts.append("%dx%d" % (rows, cols))
        left -= n
        if left < 1:
            break
    case = {"op": "step", "dtype": dtype, "shapes": ",".join(parts), "clip": 0.0}
    kind = rng.random()
    if kind < 0.25:
        return {"op": "convert", "dtype": dtype, "shapes": case["shapes"]}
    if kind < 0.6:
        case["clip"] = math.exp(rng.uniform(-3.0, 3.0))
        if dtype == "bf16" and rng.random() < 0.4:
            case["matrices"], case["width"] = rng.randint(1, 12), rng.choice([256, 384, 640, 768, 1000])
    return case


def _shapes(case):
    out = []
    for part in case["shapes"].split(","):
        times, _, what = part.rpartition("*")
        out += [tuple(int(d) for d in what.split("x"))] * int(times or 1)
    return out


class _Layout:
    """Where each tensor lies in a buffer in which every tensor starts at a
    multiple of 256 elements."""

    def __init__(self, case):
        self.shapes = _shapes(case)
        self.sizes = [math.prod(s) for s in self.shapes]
        self.blocks = [-(-n // BLOCK) for n in self.sizes]
        self.starts = np.concatenate([[0], np.cumsum(self.blocks)])[:-1] * BLOCK
        self.total = int(sum(self.blocks)) * BLOCK
        self.n = sum(self.sizes)

    def where(self):
        """Positions in the buffer of the tensors' elements, one tensor after another."""
        ends = np.cumsum(self.sizes)
        shift = torch.from_numpy(self.starts - (ends - self.sizes)).cuda()
        return torch.arange(self.n, device="cuda") + torch.repeat_interleave(
            shift, torch.tensor(self.sizes, device="cuda"), output_size=self.n)

    def views(self, flat):
        return [flat[a:a + n].view(s) for a, n, s in zip(self.starts.tolist(), self.sizes, self.shapes)]


def _inputs(case, seed):
    """Weights, gradients and a running optimizer's moments, float32, in the padded layout
    (zeros between the tensors); rows of the gradient differ in size, and some are zero as those
    of tokens that a batch does not hold."""
    lay = _Layout(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    real = torch.zeros(lay.total, device="cuda")
    real[lay.where()] = 1.0

    def normal():
        return torch.randn(lay.total, generator=gen, device="cuda")

    runs = -(-lay.total // 64)
    size = torch.exp(torch.randn(runs, generator=gen, device="cuda") * 1.5 - 5.0)
    seen = torch.rand(runs, generator=gen, device="cuda") > 0.2
    size = size.repeat_interleave(64)[:lay.total]
    seen = seen.repeat_interleave(64)[:lay.total]
    w = normal().mul_(0.02).mul_(real)
    g = normal().mul_(size).mul_(seen).mul_(real)
    m = normal().mul_(size).mul_(0.3).mul_(real)
    v = normal().square_().mul_(0.5).add_(0.5).mul_(size).mul_(size).mul_(real)
    out = {"layout": lay, "w": w, "g": g, "m": m, "v": v}
    if case.get("matrices"):
        shape = (case["matrices"], case["width"], case["width"])

        def stack(std):
            return torch.randn(shape, generator=gen, device="cuda") * std
        out.update(W=stack(0.02), G=stack(1e-2), M=stack(1e-2))
    return out


def prepare(case, seed):
    x = _inputs(case, seed)
    lay, dtype = x["layout"], DTYPES[case["dtype"]]
    state = {"case": case, "layout": lay, "seed": int(seed) & 0xffffffff, "t": STEPS_TAKEN,
             "where": lay.where(), "params": x["w"].to(dtype), "grads": x["g"].to(dtype)}
    if "W" in x:
        state.update(W=x["W"].to(torch.bfloat16), G=x["G"].to(torch.bfloat16), M=x["M"])
    values = torch.stack([x["m"][state["where"]], x["v"][state["where"]]])
    if case["op"] == "convert":
        state["values"] = values
    if own:
        import matrix_aware_optimizer_muon_amd as mm
        descs = []
        if "W" in x:
            descs = [mm.tensor_desc(w, g, m) for w, g, m in zip(state["W"], state["G"], state["M"])]
        moments = [(mm.packed_moment(p), mm.packed_moment(p)) for p in lay.views(state["params"])]
        descs += [mm.adam_tensor_desc(p, g, *mv) for p, g, mv in
                  zip(lay.views(state["params"]), lay.views(state["grads"]), moments)]
        opt = mm.MuonStep(descs, mm.default_hparams(), keepalive=moments)
        opt.set_adam_step(STEPS_TAKEN)
        opt.set_rounding_seed(state["seed"])
        opt.pack_moments(values)
        if case.get("clip"):
            opt.set_max_grad_norm(case["clip"])
        state["opt"] = opt
    else:
        first = case.get("matrices") or 0       # the AdamW tensors come after the matrices
        state["tensor"] = first + torch.repeat_interleave(
            torch.arange(len(lay.blocks), device="cuda"), torch.tensor(lay.blocks, device="cuda"))
        state["group"] = (torch.arange(lay.total // 16, device="cuda").view(-1, 16)
                          - torch.repeat_interleave(torch.from_numpy(lay.starts).cuda() // 16,
                                                    torch.tensor(lay.blocks, device="cuda"))[:, None])
        state["m"] = _nearest_first(x["m"].view(-1, BLOCK))
        state["v"] = _nearest_second(x["v"].view(-1, BLOCK))
    return state


def run(state):
    case = state["case"]
    if own:
        opt = state["opt"]
        if case["op"] == "convert":
            opt.pack_moments(state["values"])
            first, second = opt.unpack_moments(torch.float32)
            return {"first": first, "second": second}
        opt.step()
        first, second = opt.unpack_moments(torch.bfloat16)
        out = {"params": state["params"], "first": first, "second": second}
        if case.get("clip"):
            out["norm"] = opt.grad_norm
        if "W" in state:
            out["matrices"], out["momentum"] = state["W"], state["M"]
        return out
    if case["op"] == "convert":
        m, v = torch.zeros_like(state["m"]).view(-1), torch.zeros_like(state["v"]).view(-1)
        m[state["where"]], v[state["where"]] = state["values"]
        state["m"], state["v"] = _nearest_first(m.view(-1, BLOCK)), _nearest_second(v.view(-1, BLOCK))
        return {"first": state["m"].view(-1)[state["where"]], "second": state["v"].view(-1)[state["where"]]}
    return _plain_step(state)


def work(case):
    lay = _Layout(case)
    if case["op"] == "convert":     # two float32 moments in, their bytes out, and the values back
        return {"bytes": lay.n * (8 + 2 + 8), "flops": lay.n * 8}
    es = 2 if case["dtype"] == "bf16" else 4
    # weight and bytes in and out, gradient in, the moments' values (2 bytes each) out
    total, flops = lay.n * (2 * es + es + 4 + 4), lay.n * 30
    if case.get("matrices"):
        k, d = case["matrices"], case["width"]
        total += k * d * d * (2 * 2 + 2 + 2 * 4)
        flops += k * NS_STEPS * 4 * d ** 3      # two symmetric products and one full one an iteration
    return {"bytes": total, "flops": flops}


# -------------------------------------------------------------- plain form

def _mix(x):
    """32-bit mixing of integers held in int64."""
    x = ((x ^ (x >> 16)) * 0x9E3779B9) & 0xffffffff
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xffffffff
    return x ^ (x >> 16)


def _words(state):
    """The 32-bit random word of each element, [blocks, 256]."""
    key = _mix(torch.tensor(state["seed"], device="cuda"))
    key = _mix((_mix(key) + state["t"]) & 0xffffffff)
    key = _mix((key + state["tensor"]) & 0xffffffff)
    group = _mix((key[:, None] + state["group"]) & 0xffffffff)
    lane = torch.arange(16, device="cuda") * 0x9E3779B9
    return ((group[:, :, None] + lane) & 0xffffffff).view(-1, BLOCK)


def _bits(x):
    return x.view(torch.int32)


def _first_scale(m):
    e = ((_bits(m.abs().amax(1, keepdim=True)) + 0x1fffff) >> 23) - 8
    return torch.exp2(e.clamp_min(9).float() - 127)


def _first_step(a):
    """The spacing of e4m3 numbers at magnitude a."""
    return torch.exp2((torch.frexp(a)[1] - 1).clamp_min(-6).double() - 3)


def _random_first(m, u):
    scale = _first_scale(m)
    a = m.abs() / scale
    step = _first_step(a)
    return ((torch.floor(a.double() / step + u) * step).float() * scale).copysign(m)


def _nearest_first(m):
    scale = _first_scale(m)
    a = m.abs() / scale
    step = _first_step(a)
    return ((torch.round(a.double() / step) * step).float() * scale).copysign(m)


def _second_value(index, bits):
    base = (((bits.amax(1, keepdim=True) + 0xfffff) >> 20) - 255).clamp_min(0)
    index = torch.maximum(index, base + 1)
    return torch.where(bits > 0, index << 20, 0).view(torch.float32)


def _random_second(v, r):
    bits = _bits(v)
    return _second_value((bits + r) >> 20, bits)


def _nearest_second(v):
    bits = _bits(v)
    base = (((bits.amax(1, keepdim=True) + 0xfffff) >> 20) - 255).clamp_min(0)
    index = torch.minimum((bits + 0x7ffff + ((bits >> 20) & 1)) >> 20, base + 255)
    return _second_value(index, bits)


def _muon(W, G, M):
    """One Muon step of a stack of square matrices, in float32."""
    g = G * (1 - MUON_MU)
    M.mul_(MUON_MU).add_(g)
    x = M * MUON_MU + g
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + MUON_EPS)
    for _ in range(NS_STEPS):
        a = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = NS_A * x + torch.bmm(NS_B * a + NS_C * torch.bmm(a, a), x)
    w = W.float()
    W.copy_(w - MUON_LR * MUON_DECAY * w - MUON_LR * x)


def _plain_step(state):
    case, out = state["case"], {}
    state["t"] += 1
    t = state["t"]
    g = state["grads"].float()
    G = state["G"].float() if "G" in state else None
    if case.get("clip"):
        total = g.double().square().sum()
        if G is not None:
            total = total + G.double().square().sum()
        norm = total.sqrt()
        factor = torch.clamp(case["clip"] / norm, max=1.0).float()
        out["norm"] = torch.stack([norm.float(), factor])
        g = g * factor
        G = G * factor if G is not None else None
    if G is not None:
        _muon(state["W"], G, state["M"])
        out["matrices"], out["momentum"] = state["W"], state["M"]
    g = g.view(-1, BLOCK)
    m = BETA1 * state["m"] + (1 - BETA1) * g
    v = BETA2 * state["v"] + ((1 - BETA2) * g) * g
    w = state["params"].float().view(-1, BLOCK)
    den = v.sqrt() * (1 / math.sqrt(1 - BETA2 ** t)) + EPS
    w = w - LR * DECAY * w - LR * (m * (1 / (1 - BETA1 ** t)) / den)
    state["params"].copy_(w.view(-1))
    r = _words(state)
    state["m"] = _random_first(m, (r >> 12).double() / 2 ** 20)
    state["v"] = _random_second(v, (r & 0xfffff).int())
    out["params"] = state["params"]
    out["first"] = state["m"].view(-1)[state["where"]].bfloat16()
    out["second"] = state["v"].view(-1)[state["where"]].bfloat16()
    return out


# --------------------------------------------------- definition in 64 bits

def _hash32(x):
    with np.errstate(over="ignore"):
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0x9E3779B9)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0xBB67AE85)
    return x ^ (x >> np.uint32(16))


def _element_words(seed, t, tensor, n):
    one = lambda k: np.array([k & 0xffffffff], np.uint32)  # noqa: E731
    key = _hash32(_hash32(_hash32(_hash32(one(seed))) + one(t)) + one(tensor))
    group = _hash32(key + np.arange(-(-n // 16), dtype=np.uint32))
    words = group[:, None] + np.arange(16, dtype=np.uint32) * np.uint32(0x9E3779B9)
    return torch.from_numpy(words.reshape(-1)[:n].astype(np.int64)).cuda()


def _grid_first():
    """The non-negative e4m3 numbers in rising order."""
    sub = [k * 2.0 ** -9 for k in range(8)]
    return torch.tensor(sub + [(1 + k / 8) * 2.0 ** e for e in range(-6, 9) for k in range(8)][:-1],
                        dtype=torch.float64, device="cuda")


def _grid_second():
    """The float32 numbers whose lower 20 bits are zero, by their index, and infinity."""
    sub = [k / 8 * 2.0 ** -126 for k in range(8)]
    return torch.tensor(sub + [(1 + k / 8) * 2.0 ** (e - 127) for e in range(1, 255) for k in range(8)] + [math.inf],
                        dtype=torch.float64, device="cuda")


def _between(grid, a, u):
    """Each a's lower neighbour's place in the grid, or the upper one's where its share of the way there and u
    make one; u None: the nearer one, ties to the even place."""
    low = (torch.searchsorted(grid, a, right=True) - 1).clamp(max=grid.numel() - 2)
    share = (a - grid[low]) / (grid[low + 1] - grid[low])
    up = share + u >= 1 if u is not None else (share > 0.5) | ((share == 0.5) & (low % 2 == 1))
    return low + up.long()


def _blocks_max(x):
    pad = -x.numel() % BLOCK
    return torch.cat([x, x.new_zeros(pad)]).view(-1, BLOCK).amax(1)


def _per_element(x, n):
    return x.repeat_interleave(BLOCK)[:n]


def _hold_first(m, u):
    big = _blocks_max(m.abs())
    mant, e = torch.frexp(big)                  # big = mant 2^e; a mantissa above 0.875 (1.75) needs one binade more
    k = (e - 1 + (mant > 0.875).int() - 8).clamp_min(9 - 127)
    scale = torch.exp2(_per_element(k.double(), m.numel()))
    grid = _grid_first()
    return torch.sign(m) * grid[_between(grid, m.abs() / scale, u)] * scale


def _hold_second(v, u):
    grid = _grid_second()
    top = torch.searchsorted(grid, _blocks_max(v), right=False)     # the first one not below the largest
    base = _per_element((top - 255).clamp_min(0), v.numel())
    place = torch.minimum(torch.maximum(_between(grid, v, u), base + 1), base + 255)
    return torch.where(v > 0, grid[place], 0.0)


def exact(case, seed):
    x = _inputs(case, seed)
    lay, dtype, t = x["layout"], DTYPES[case["dtype"]], STEPS_TAKEN + 1
    cut = lambda name: [z.reshape(-1) for z in lay.views(x[name])]  # noqa: E731
    if case["op"] == "convert":
        first = [_hold_first(m.double(), None) for m in cut("m")]
        second = [_hold_second(v.double(), None) for v in cut("v")]
        return {"first": torch.cat(first), "second": torch.cat(second)}
    out, factor = {}, 1.0
    grads = [g.to(dtype).double() for g in cut("g")]
    if "G" in x:
        W, G, M = (x["W"].bfloat16().double(), x["G"].bfloat16().double(), x["M"].double())
    if case.get("clip"):
        total = sum(float((g * g).sum()) for g in grads) + (float((G * G).sum()) if "G" in x else 0.0)
        factor = min(1.0, case["clip"] / math.sqrt(total))
        out["norm"] = torch.tensor([math.sqrt(total), factor], dtype=torch.float64)
    if "G" in x:
        G = (1 - MUON_MU) * factor * G
        M = MUON_MU * M + G
        u = MUON_MU * M + G
        u = u / (torch.linalg.matrix_norm(u)[:, None, None] + MUON_EPS)
        for _ in range(NS_STEPS):
            a = u @ u.mT.contiguous()
            u = NS_A * u + NS_B * (a @ u) + NS_C * (a @ (a @ u))
        out["matrices"], out["momentum"] = W * (1 - MUON_LR * MUON_DECAY) - MUON_LR * u, M
    first, second = [], []
    params = torch.zeros(lay.total, dtype=torch.float64, device="cuda")
    for k, (w, g, m, v) in enumerate(zip(cut("w"), grads, cut("m"), cut("v"))):
        n = g.numel()
        g = g * factor
        m = BETA1 * _hold_first(m.double(), None) + (1 - BETA1) * g
        v = BETA2 * _hold_second(v.double(), None) + (1 - BETA2) * g * g
        w = w.to(dtype).double()
        den = torch.sqrt(v / (1 - BETA2 ** t)) + EPS
        start = int(lay.starts[k])
        params[start:start + n] = w - LR * (DECAY * w + m / (1 - BETA1 ** t) / den)
        word = _element_words(int(seed), t, k + (case.get("matrices") or 0), n)
        first.append(_hold_first(m, (word >> 12).double() / 2 ** 20))
        second.append(_hold_second(v, (word & 0xfffff).double() / 2 ** 20))
    out["params"] = params
    out["first"], out["second"] = torch.cat(first), torch.cat(second)
    return out
