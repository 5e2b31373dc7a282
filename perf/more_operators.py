"""Cases that time the operators of an adapted head: low-rank adapters beside the
shared projection (forward and backward), the AdamW step over many tensors that
follows the gradients, and beam search over the logits.

``run`` computes them in elementary torch operations (``own`` false) or through
the package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32       # values that share a scale of the 8-bit states
ALIGN = 128      # every tensor's states start at a multiple of this many elements
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ELEM = {"bf16": 2, "fp32": 4}
BETAS, EPS, DECAY, LR, STEP, SEED = (0.9, 0.999), 1e-8, 0.01, 1e-3, 40, 20240917
MAX_NORM = 1.0


def listed():
    return [
        # one decoding step of eight sequences, each with an adapter of its own, over the
        # repository's largest classifier
        dict(name="lora_decode", op="lora_fwd", M=8, H=4096, V=131072, n=8, r=16, dtype="bf16",
             base=False, order="mixed"),
        # a serving batch beside logits that another product (a microscaled head) has made
        dict(name="lora_beside", op="lora_fwd", M=64, H=4096, V=128256, n=16, r=16, dtype="bf16",
             base=True, order="mixed"),
        # the prompts of a few requests, token after token
        dict(name="lora_prompts", op="lora_fwd", M=2048, H=4096, V=32000, n=4, r=16, dtype="bf16",
             base=False, order="runs"),
        # 61 sequences over the repository's odd vocabulary, FP32 logits, the smallest rank
        dict(name="lora_odd_vocab", op="lora_fwd", M=61, H=2304, V=256003, n=5, r=8, dtype="fp32",
             base=False, order="mixed"),
        # fine-tuning two adapters at once through the frozen classifier
        dict(name="lora_train", op="lora_bwd", M=2600, H=2304, V=32000, n=2, r=32, dtype="bf16",
             base=False, order="runs"),
        # the adapters' gradients alone, FP32 gradient of the logits, odd everything
        dict(name="lora_train_odd", op="lora_bwd", M=1021, H=2304, V=4099, n=3, r=16,
             dtype="fp32", base=True, order="mixed"),
        # the adapters of one fine-tuning run: many small FP32 tensors, clipped, latency
        dict(name="adamw_adapters", op="adamw", sizes="65536,512000," * 7 + "65536,512000",
             dtype="fp32", gdtype="fp32", bits=32, master=False, clip=True),
        # a classifier in BF16 with FP32 masters, and the norm before it
        dict(name="adamw_head", op="adamw", sizes="131072000,4096", dtype="bf16", gdtype="bf16",
             bits=32, master=True, clip=True),
        # the same classifier with 8-bit states, and tensors of odd sizes beside it
        dict(name="adamw_head_8bit", op="adamw", sizes="131072000,4096,1,2305,100003",
             dtype="bf16", gdtype="bf16", bits=8, master=False, clip=False),
        # one request with four beams: latency
        dict(name="beam_one", op="beam", B=1, K=4, V=32000, n_out=4, dtype="bf16", ended=False,
             layers=0, row=0, sigma=4.0),
        # a batch of requests with eight beams each, their histories and caches reordered
        dict(name="beam_batch", op="beam", B=16, K=8, V=128256, n_out=8, dtype="bf16",
             ended=False, layers=4, row=262144, sigma=4.0),
        # FP32 logits over the odd vocabulary, twice as many candidates as beams, some beams ended
        dict(name="beam_odd_vocab", op="beam", B=5, K=5, V=256003, n_out=10, dtype="fp32",
             ended=True, layers=1, row=5003, sigma=3.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lora_fwd", "lora_fwd", "lora_bwd", "adamw", "adamw", "beam", "beam"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("lora_fwd", "lora_bwd"):
        H = _log_int(rng, 64, 8192) // 8 * 8
        V = _log_int(rng, 500, 131072 if op == "lora_fwd" else 32000)
        top = 2048 * 4096 * 32000 // H // V if op == "lora_fwd" else 2600 * 2304 * 32000 // H // V
        M = _log_int(rng, 1, max(1, min(2048 if op == "lora_fwd" else 2600, top // 2)))
        return dict(op=op, M=M, H=H, V=V, n=_log_int(rng, 1, 32), r=8 * _log_int(rng, 1, 8),
                    dtype=dtype, base=rng.random() < 0.4, order=rng.choice(["mixed", "runs"]))
    if op == "adamw":
        total, sizes = _log_int(rng, 1000, 60000000), []
        for _ in range(_log_int(rng, 1, 40)):
            sizes.append(_log_int(rng, 1, max(2, total // 2)))
            total = max(2, total - sizes[-1])
        return dict(op=op, sizes=",".join(str(s) for s in sizes), dtype=dtype,
                    gdtype=rng.choice(["bf16", "fp32"]), bits=rng.choice([8, 32]),
                    master=dtype == "bf16" and rng.random() < 0.5, clip=rng.random() < 0.5)
    V = _log_int(rng, 500, 262144)
    K = _log_int(rng, 1, 16)
    B = _log_int(rng, 1, max(1, min(64, 16 * 8 * 128256 // V // K)))
    return dict(op=op, B=B, K=K, V=V, n_out=rng.choice([K, 2 * K]), dtype=dtype,
                ended=rng.random() < 0.4, layers=rng.choice([0, 1, 2]),
                row=_log_int(rng, 10, 100000), sigma=round(rng.uniform(1.5, 5.0), 2))


# ---- inputs -------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _adapters(g, M, n, order):
    """An adapter per token: -1 for none, in runs as prompts come, or mixed as decoding does."""
    if order == "runs":
        cut = torch.sort(torch.randint(0, M + 1, (n,), generator=g, device="cuda")).values
        pos = torch.arange(M, device="cuda")
        return (torch.searchsorted(cut, pos, right=True) - 1).to(torch.int32)
    return torch.randint(-1, n, (M,), generator=g, device="cuda").to(torch.int32)


def _pow2(e):
    """2^e in FP32 from its bits, for integers e (clamped to the normal range)."""
    return ((e.to(torch.int32).clamp(-126, 127) + 127) << 23).view(torch.float32)


def _layout(case):
    """(sizes, offsets, total): where each tensor's states lie in the flat buffers."""
    sizes = [int(s) for s in case["sizes"].split(",")]
    offs, at = [], 0
    for s in sizes:
        offs.append(at)
        at += (s + ALIGN - 1) // ALIGN * ALIGN
    return sizes, offs, at


def _bytes_of(v):
    """FP32 (multiple of 32) to E4M3 codes and scale bytes, to nearest."""
    b = v.view(-1, BLOCK)
    e = _scale_exponent(b)
    x = b * _pow2(-e)
    _, ex = torch.frexp(x)
    ex = torch.clamp(ex - 1, min=-6)
    k = torch.round(x.abs() * _pow2(3 - ex)).to(torch.int32)  # a carry to 16 is the next binade
    code = ((ex + 6) << 3) + k
    code = code | ((x < 0).to(torch.int32) << 7)
    return code.to(torch.uint8).view(-1), (e.view(-1) + 127).to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    st = dict(case=case)
    if op.startswith("lora"):
        M, H, V, n, r = (case[k] for k in ("M", "H", "V", "n", "r"))
        st["x"] = _randn(g, (M, H), torch.bfloat16)
        st["a"] = _randn(g, (n, r, H), torch.bfloat16, H ** -0.5)
        st["b"] = _randn(g, (n, V, r), torch.bfloat16, r ** -0.5)
        st["scale"] = torch.rand(n, generator=g, device="cuda") * 1.5 + 0.5
        st["adapter"] = _adapters(g, M, n, case["order"])
        st["w"] = st["base"] = None
        if op == "lora_bwd":
            st["dy"] = _randn(g, (M, V), dt, 0.01)
            if case["base"]:
                st["base"] = _randn(g, (M, H), torch.bfloat16, 0.01)
        elif case["base"]:
            st["base"] = _randn(g, (M, V), dt, 2.0)
        if not case["base"]:
            st["w"] = _randn(g, (V, H), torch.bfloat16, 2.0 * H ** -0.5)
        if own:
            import vocabulary_cross_entropy_amd as vce
            st["ws"] = (vce.lora_backward_workspace(M, H, V, n, r, dt) if op == "lora_bwd"
                        else vce.lora_forward_workspace(M, H, V, n, r))
    elif op == "adamw":
        sizes, offs, total = _layout(case)
        gd = DTYPES[case["gdtype"]]
        p32 = [torch.randn(s, generator=g, device="cuda") * 0.02 for s in sizes]
        st["p"] = [p.to(dt) for p in p32]
        st["g"] = [_randn(g, (s,), gd, 1e-3) for s in sizes]
        m = torch.zeros(total, device="cuda")
        root = torch.zeros(total, device="cuda")
        master = torch.zeros(total if case["master"] else 0, device="cuda")
        for p, s, o in zip(p32, sizes, offs):
            m[o:o + s] = torch.randn(s, generator=g, device="cuda") * 3e-4
            root[o:o + s] = 1e-3 * torch.exp(torch.randn(s, generator=g, device="cuda") * 0.7)
            if case["master"]:
                master[o:o + s] = p
        if case["bits"] == 8:
            st["m"], st["ms"] = _bytes_of(m)
            st["v"], st["vs"] = _bytes_of(root)
        else:
            st["m"], st["v"], st["ms"], st["vs"] = m, root * root, None, None
        st["master"] = master
        if own:
            import vocabulary_cross_entropy_amd as vce
            s = st["state"] = vce.adamw_state(st["p"], bits=case["bits"], master=case["master"])
            for name, t in (("m", st["m"]), ("v", st["v"]), ("m_scales", st["ms"]),
                            ("v_scales", st["vs"])):
                if t is not None:
                    getattr(s, name).copy_(t)
            if case["master"]:
                s.master.copy_(master)
    else:
        B, K, V = case["B"], case["K"], case["V"]
        z = torch.randn((B * K, V), generator=g, device="cuda") * case["sigma"]
        # a few likely continuations in every row
        top = torch.randint(0, V, (B * K, 8), generator=g, device="cuda")
        z.scatter_(1, top, torch.randn((B * K, 8), generator=g, device="cuda") * 2 +
                   3.5 * case["sigma"])
        st["z"] = z.to(dt).view(B, K, V)
        st["scores"] = -5.0 * torch.rand((B, K), generator=g, device="cuda") - 10.0
        st["ended"] = None
        if case["ended"]:
            st["ended"] = torch.rand((B, K), generator=g, device="cuda") < 0.25
        st["states"] = [torch.randint(0, V, (B, K, 37), generator=g, device="cuda")]
        for _ in range(case["layers"]):
            st["states"].append(_randn(g, (B, K, case["row"]), torch.bfloat16))
        if own:
            import vocabulary_cross_entropy_amd as vce
            st["ws"] = vce.beam_workspace(B, K, V)
    return st


# ---- plain forms -------------------------------------------------------------------

def _lora_forward_plain(st):
    c = st["case"]
    x, b = st["x"].float(), st["b"].float()
    y = st["base"].float() if st["w"] is None else x @ st["w"].float().t()
    # every adapter's share for every token, kept where the token has it
    for k, a in enumerate(st["a"].float()):
        mine = (st["adapter"] == k).unsqueeze(1)
        s = torch.where(mine, (x @ a.t()) * st["scale"][k], 0.0)
        y = y + s @ b[k].t()
    return [y.to(DTYPES[c["dtype"]])]


def _lora_backward_plain(st):
    x, a, b, dy = st["x"].float(), st["a"].float(), st["b"].float(), st["dy"].float()
    dx = st["base"].float() if st["w"] is None else dy @ st["w"].float()
    da, db = torch.empty_like(a), torch.empty_like(b)
    for k in range(a.shape[0]):
        mine = (st["adapter"] == k).unsqueeze(1)
        s = torch.where(mine, (x @ a[k].t()) * st["scale"][k], 0.0)
        ds = torch.where(mine, (dy @ b[k]) * st["scale"][k], 0.0)
        dx = dx + ds @ a[k]
        da[k] = ds.t() @ x
        db[k] = dy.t() @ s
    return [dx.to(torch.bfloat16), da, db]


def _scale_exponent(b):
    """Exponent of the least power of two s with max |b| <= 448 s over blocks (n, 32)."""
    m, e = torch.frexp(b.abs().amax(1, keepdim=True))
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.clamp(torch.where(m == 0, torch.full_like(e, -127), e), -127, 127)


def _values_of(q, s):
    code = q.to(torch.int32) & 127
    ex, man = code >> 3, code & 7
    v = torch.where(ex > 0, (man + 8).float() * _pow2(ex - 10), man.float() * 2.0 ** -9)
    v = torch.where(q >= 128, -v, v)
    return (v.view(-1, BLOCK) * _pow2(s.to(torch.int32) - 127).unsqueeze(1)).view(-1)


def _mix(x):
    """32 bits to 32 bits, one to one, in 64-bit integers."""
    x = ((x ^ (x >> 16)) * 0x9E3779B9) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x6A09E667) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random_bits(n, seed, step, device):
    """32 random bits for each of the flat places 0 .. n - 1."""
    lo, hi = (torch.tensor(t, dtype=torch.int64) for t in (seed & 0xFFFFFFFF, seed >> 32))
    key = _mix((_mix(lo ^ _mix(hi)) + step) & 0xFFFFFFFF)
    i = torch.arange(n, device=device)
    return _mix((i & 0xFFFFFFFF) ^ _mix((key.to(device) + (i >> 32)) & 0xFFFFFFFF))


def _round_random(v, bits16, keep):
    """FP32 to E4M3 values with a scale per 32, up or down by 16 random bits; nothing but zero
    becomes zero with `keep`.  As codes and scale bytes."""
    b = v.view(-1, BLOCK)
    e = _scale_exponent(b)
    x = b * _pow2(-e)
    _, ex = torch.frexp(x)
    ex = torch.clamp(ex - 1, min=-6)
    t = x.abs() * _pow2(3 - ex)
    k = torch.floor(t)
    k = k + ((t - k) * 65536.0 > bits16.view(-1, BLOCK).float()).float()
    if keep:
        k = torch.where((x != 0) & (k == 0), 1.0, k)
    code = ((ex + 6) << 3) + k.to(torch.int32)
    code = code | ((x < 0).to(torch.int32) << 7)
    return code.to(torch.uint8).view(-1), (e.view(-1) + 127).to(torch.uint8)


def _adamw_plain(st):
    c = st["case"]
    sizes, offs, total = _layout(c)
    (b1, b2), dt = BETAS, DTYPES[c["dtype"]]
    bc1, bc2 = 1.0 - b1 ** STEP, 1.0 - b2 ** STEP
    scale, out = None, []
    if c["clip"]:
        norm = torch.sqrt(sum((g.double() ** 2).sum() for g in st["g"]))
        scale = torch.where(norm > MAX_NORM, MAX_NORM / norm, 1.0).float()
        out.append(norm.float())
    g = torch.zeros(total, device=st["m"].device)
    for t, s, o in zip(st["g"], sizes, offs):
        g[o:o + s] = t.float() if scale is None else t.float() * scale
    if c["bits"] == 8:
        m, root = _values_of(st["m"], st["ms"]), _values_of(st["v"], st["vs"])
        v = root * root
    else:
        m, v = st["m"], st["v"]
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    step = (LR / bc1) * m / (torch.sqrt(v) / math.sqrt(bc2) + EPS)
    for k, (s, o) in enumerate(zip(sizes, offs)):
        p = st["master"][o:o + s] if c["master"] else st["p"][k].float()
        p = p * (1.0 - LR * DECAY) - step[o:o + s]
        if c["master"]:
            st["master"][o:o + s] = p
        st["p"][k].copy_(p.to(dt))
    if c["bits"] == 8:
        r = _random_bits(total, SEED, STEP, g.device)
        st["m"], st["ms"] = _round_random(m, r & 0xFFFF, False)
        st["v"], st["vs"] = _round_random(torch.sqrt(v), r >> 16, True)
        out += [_values_of(st["m"], st["ms"]).bfloat16(), _values_of(st["v"], st["vs"]).bfloat16()]
    else:
        st["m"], st["v"] = m, v
        out += [m, v]
    return out + st["p"] + ([st["master"]] if c["master"] else [])


def _beam_plain(st):
    c = st["case"]
    B, K, V = st["z"].shape
    z = st["z"].double()
    m = z.amax(2, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(2, keepdim=True))
    val = st["scores"].double().unsqueeze(2) + (z - lse)
    if st["ended"] is not None:  # an ended beam goes on as it is, with the end token
        only = torch.full_like(val, -math.inf)
        only[:, :, 0] = st["scores"].double()
        val = torch.where(st["ended"].unsqueeze(2), only, val)
    val, at = torch.sort(val.view(B, K * V), dim=1, descending=True, stable=True)
    n = c["n_out"]
    parent = (at[:, :n] // V).to(torch.int32)
    for t in st["states"]:
        rows = parent[:, :K].long().view(B, K, *([1] * (t.dim() - 2))).expand(t.shape)
        t.copy_(torch.gather(t, 1, rows))
    return [val[:, :n].float(), parent, at[:, :n] % V] + st["states"]


def _run_plain(st):
    op = st["case"]["op"]
    if op == "lora_fwd":
        return _lora_forward_plain(st)
    if op == "lora_bwd":
        return _lora_backward_plain(st)
    return _adamw_plain(st) if op == "adamw" else _beam_plain(st)


def _run_own(st):
    import vocabulary_cross_entropy_amd as vce
    c = st["case"]
    op = c["op"]
    if op == "lora_fwd":
        return [vce.lora_forward(st["x"], st["a"], st["b"], st["adapter"], st["w"],
                                 base=st["base"], scale=st["scale"], dtype=DTYPES[c["dtype"]],
                                 workspace=st["ws"])]
    if op == "lora_bwd":
        return list(vce.lora_backward(st["dy"], st["x"], st["a"], st["b"], st["adapter"],
                                      st["w"], dx_base=st["base"], scale=st["scale"],
                                      workspace=st["ws"]))
    if op == "adamw":
        s, out, scale = st["state"], [], None
        if c["clip"]:
            norm, scale = vce.grad_norm(st["g"], MAX_NORM)
            out.append(norm)
        vce.adamw_step(st["p"], st["g"], s, LR, STEP, betas=BETAS, eps=EPS, weight_decay=DECAY,
                       grad_scale=scale, seed=SEED)
        if c["bits"] == 8:
            out += [vce.mx_dequantize(q.view(-1, ALIGN), b.view(-1, ALIGN // BLOCK),
                                      "e4m3").view(-1)
                    for q, b in ((s.m, s.m_scales), (s.v, s.v_scales))]
        else:
            out += [s.m, s.v]
        return out + st["p"] + ([s.master] if c["master"] else [])
    score, parent, token = vce.beam_step(st["z"], st["scores"], c["n_out"], ended=st["ended"],
                                         end_token=0, workspace=st["ws"])
    vce.beam_reorder(st["states"], parent[:, :c["K"]])
    return [score, parent, token] + st["states"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definitions in 64 bits ------------------------------------------------------

def _exact_lora(st, backward):
    x, a, b = st["x"].double(), st["a"].double(), st["b"].double()
    n, M = a.shape[0], x.shape[0]
    # scale of adapter k where token i has it: y = base + sum_k diag(on[k]) x A_k^T B_k^T
    on = torch.zeros((n, M), dtype=torch.float64, device=x.device)
    for i, k in enumerate(st["adapter"].tolist()):
        if k >= 0:
            on[k, i] = float(st["scale"][k])
    if not backward:
        y = st["base"].double() if st["w"] is None else x @ st["w"].double().t()
        for k in range(n):
            rows = torch.nonzero(on[k]).view(-1)
            y[rows] += on[k, rows].unsqueeze(1) * (x[rows] @ a[k].t() @ b[k].t())
        return [y]
    dy = st["dy"].double()
    dx = st["base"].double() if st["w"] is None else dy @ st["w"].double()
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for k in range(n):
        rows = torch.nonzero(on[k]).view(-1)
        gx = on[k, rows].unsqueeze(1) * (dy[rows] @ b[k])
        dx[rows] += gx @ a[k]
        da[k] = gx.t() @ x[rows]
        db[k] = (on[k, rows].unsqueeze(1) * dy[rows]).t() @ (x[rows] @ a[k].t())
    return [dx, da, db]


def _exact_decode(q, s):
    """Values of E4M3 codes with scales, by a table of all codes."""
    table = []
    for code in range(256):
        ex, man = (code >> 3) & 15, code & 7
        f = man / 8 * 2.0 ** -6 if ex == 0 else (1 + man / 8) * 2.0 ** (ex - 7)
        table.append(-f if code >> 7 else f)
    t = torch.tensor(table, dtype=torch.float64, device=q.device)[q.long()]
    return t * torch.exp2(s.double() - 127).repeat_interleave(BLOCK)


def _exact_random(n, seed, step):
    def mix(x):
        x = (x ^ (x >> np.uint64(16))) * np.uint64(0x9E3779B9) & np.uint64(0xFFFFFFFF)
        x = (x ^ (x >> np.uint64(15))) * np.uint64(0x6A09E667) & np.uint64(0xFFFFFFFF)
        return x ^ (x >> np.uint64(16))
    word = np.uint64(0xFFFFFFFF)
    k = mix(np.array([seed & 0xFFFFFFFF], np.uint64) ^ mix(np.array([seed >> 32], np.uint64)))
    k = mix((k + np.uint64(step)) & word)
    i = np.arange(n, dtype=np.uint64)
    return mix((i & word) ^ mix((k + (i >> np.uint64(32))) & word))


def _exact_round(v, r16, keep):
    """Neighbours on the grid of each block's scale by division, one of them by r16."""
    b = v.view(-1, BLOCK)
    amax = b.abs().amax(1, keepdim=True)
    s = torch.exp2(torch.ceil(torch.log2(torch.where(amax > 0, amax, 1.0) / 448.0)))
    s = torch.where(s * 448.0 < amax, s * 2, s)
    a = b.abs() / s
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.where(a > 0, a, 1.0))), -6) - 3)
    lo = torch.floor(a / step)
    up = (a / step - lo) > r16.view(-1, BLOCK) / 65536.0
    k = lo + up
    if keep:
        k = torch.where((a > 0) & (k == 0), 1.0, k)
    return (torch.sign(b) * k * step * s).view(-1)


def _exact_adamw(st):
    c = st["case"]
    sizes, offs, total = _layout(c)
    dev = st["m"].device
    b1, b2 = BETAS
    g = torch.zeros(total, dtype=torch.float64, device=dev)
    p = torch.zeros(total, dtype=torch.float64, device=dev)
    for k, (s, o) in enumerate(zip(sizes, offs)):
        g[o:o + s] = st["g"][k].double()
        p[o:o + s] = st["p"][k].double()
    if c["master"]:
        p = st["master"].double()
    out = []
    if c["clip"]:
        norm = float(torch.linalg.vector_norm(g))
        out.append(torch.tensor(norm, dtype=torch.float64, device=dev))
        g = g * min(1.0, MAX_NORM / norm)
    if c["bits"] == 8:
        m, v = _exact_decode(st["m"], st["ms"]), _exact_decode(st["v"], st["vs"]) ** 2
    else:
        m, v = st["m"].double(), st["v"].double()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    p = p - LR * (DECAY * p + m / (1 - b1 ** STEP) /
                  (torch.sqrt(v / (1 - b2 ** STEP)) + EPS))
    if c["bits"] == 8:
        r = torch.from_numpy(_exact_random(total, SEED, STEP).astype(np.int64)).to(dev)
        out += [_exact_round(m, (r % 65536).double(), False),
                _exact_round(torch.sqrt(v), (r // 65536).double(), True)]
    else:
        out += [m, v]
    out += [p[o:o + s] for s, o in zip(sizes, offs)]
    return out + ([p] if c["master"] else [])


def _exact_beam(st):
    c = st["case"]
    B, K, V = st["z"].shape
    z = st["z"].float().cpu().numpy()
    s0 = st["scores"].cpu().numpy().astype(np.float64)
    ended = None if st["ended"] is None else st["ended"].cpu().numpy()
    n = c["n_out"]
    score = np.zeros((B, n))
    parent, token = np.zeros((B, n), np.int32), np.zeros((B, n), np.int64)
    for q in range(B):
        best = []
        for k in range(K):
            if ended is not None and ended[q, k]:
                best.append((-s0[q, k], k, 0))
                continue
            row = z[q, k].astype(np.float64)
            top = np.argpartition(-row, n)[:n] if n < V else np.arange(V)
            top = np.flatnonzero(row >= row[top].min())
            lse = row.max() + math.log(np.exp(row - row.max()).sum())
            best += [(-(s0[q, k] + (row[v] - lse)), k, int(v)) for v in top]
        for i, (v, k, t) in enumerate(sorted(best)[:n]):
            score[q, i], parent[q, i], token[q, i] = -v, k, t
    states = []
    for t in st["states"]:
        h = t.clone()
        for q in range(B):
            for k in range(K):
                h[q, k] = t[q, int(parent[q, k])]
        states.append(h if t.dtype == torch.int64 else h.double())
    return [torch.from_numpy(score), torch.from_numpy(parent), torch.from_numpy(token)] + states


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("lora"):
        return _exact_lora(st, case["op"] == "lora_bwd")
    return _exact_adamw(st) if case["op"] == "adamw" else _exact_beam(st)


def work(case):
    op, es = case["op"], ELEM[case["dtype"]]
    if op.startswith("lora"):
        M, H, V, n, r = (case[k] for k in ("M", "H", "V", "n", "r"))
        used = min(n, M)
        ab = used * r * (H + V) * 2
        if op == "lora_fwd":
            shared = M * V * es if case["base"] else V * H * 2
            return dict(bytes=M * H * 2 + ab + shared + M * V * es,
                        flops=2 * M * r * (H + V) + (0 if case["base"] else 2 * M * H * V))
        shared = M * H * 2 if case["base"] else V * H * 2
        return dict(bytes=M * V * es + 2 * M * H * 2 + ab + shared + n * r * (H + V) * 4,
                    flops=6 * M * r * (H + V) + (0 if case["base"] else 2 * M * H * V))
    if op == "adamw":
        n = sum(int(s) for s in case["sizes"].split(","))
        state = 4 * 8 if case["bits"] == 32 else 4 * (1 + 1 / BLOCK)
        state = state / 2 if case["bits"] == 32 else state
        per = 2 * es + ELEM[case["gdtype"]] * (2 if case["clip"] else 1) + state
        per += (8 - es) if case["master"] else 0  # the master is read in the parameter's place
        return dict(bytes=int(n * per), flops=16 * n)
    n = case["B"] * case["K"] * case["V"]
    moved = case["B"] * (case["K"] - 1) * (37 * 8 + case["layers"] * case["row"] * 2)
    return dict(bytes=n * es + 2 * moved, flops=4 * n)
