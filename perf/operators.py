"""Cases that time the operators around the vocabulary head.

Four operators: the residual + RMS norm that makes the head's input (forward,
forward into microscaled 8 bits, backward), the microscaled quantisation, the
head's product over microscaled operands, and the draw of a token from the
logits.  ``run`` computes them in elementary torch operations (``own`` false)
or through the package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
# per format: mantissa bits, least exponent of a normal value, largest value
FORMATS = {"e4m3": (3, -6, 448.0), "e2m1": (1, 0, 6.0)}
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ELEM = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # one decoding step of eight sequences: 8-bit head input, latency only
        dict(name="rms_mx8_decode", op="rms_mx8", M=8, H=4096, dtype="bf16", residual=True,
             offset=0.0),
        # a training step's tokens at the repository's larger linear workload (H = 2304,
        # weights stored as w - 1)
        dict(name="rms_train_fwd", op="rms_fwd", M=16384, H=2304, dtype="bf16", residual=True,
             offset=1.0),
        # the same step's backward, with the gradient of the residual stream added
        dict(name="rms_train_bwd", op="rms_bwd", M=16384, H=2304, dtype="bf16", residual=True,
             offset=1.0),
        # FP32 training of a small model whose width is no multiple of a vector
        dict(name="rms_odd_bwd", op="rms_bwd", M=1021, H=2305, dtype="fp32", residual=False,
             offset=0.0),
        # a head's weights to 4 bits and back, once when a checkpoint is loaded
        dict(name="mx4_weights", op="mx_round", rows=32000, H=4096, dtype="bf16", fmt="e2m1"),
        # FP32 activations of an odd number of rows to 8 bits and back
        dict(name="mx8_odd_rows", op="mx_round", rows=333, H=2304, dtype="fp32", fmt="e4m3"),
        # one decoding step of eight sequences through the 4-bit head
        dict(name="head_decode", op="mx_logits", M=8, H=4096, V=131072, x_fmt="e4m3",
             w_fmt="e2m1", dtype="bf16"),
        # 61 sequences, the repository's odd vocabulary, 4 bits on both sides, FP32 logits
        dict(name="head_batch_odd_vocab", op="mx_logits", M=61, H=2304, V=256003, x_fmt="e2m1",
             w_fmt="e2m1", dtype="fp32"),
        # log-probabilities of a prompt: every token's logits
        dict(name="head_prompt", op="mx_logits", M=4096, H=4096, V=32000, x_fmt="e4m3",
             w_fmt="e2m1", dtype="bf16"),
        # one sequence, all three filters: latency
        dict(name="sample_one", op="sample", N=1, V=128256, dtype="bf16", mode="filters",
             sigma=4.0),
        # a serving batch whose requests ask for different things
        dict(name="sample_batch", op="sample", N=256, V=128256, dtype="bf16", mode="mixed",
             sigma=4.0),
        # plain temperature over a large odd vocabulary, FP32 logits
        dict(name="sample_temperature", op="sample", N=61, V=256003, dtype="fp32",
             mode="temperature", sigma=3.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_bwd", "rms_mx8", "mx_round", "mx_logits", "mx_logits",
                     "sample", "sample"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("rms_fwd", "rms_bwd", "rms_mx8"):
        H = _log_int(rng, 64, 16384)
        if op == "rms_mx8" or rng.random() < 0.7:
            H = max(32, H // 32 * 32)
        M = _log_int(rng, 1, max(1, min(16384, 16384 * 2304 // H)))
        return dict(op=op, M=M, H=H, dtype=dtype, residual=rng.random() < 0.7,
                    offset=rng.choice([0.0, 1.0]))
    if op == "mx_round":
        H = max(32, _log_int(rng, 64, 16384) // 32 * 32)
        return dict(op=op, rows=_log_int(rng, 1, 32000 * 4096 // H // 2), H=H, dtype=dtype,
                    fmt=rng.choice(["e4m3", "e2m1"]))
    if op == "mx_logits":
        H = max(64, _log_int(rng, 64, 8192) // 32 * 32)
        V = _log_int(rng, 1000, min(262144, 131072 * 4096 // H))
        M = _log_int(rng, 1, max(1, min(4096, 4096 * 32000 // V // 2)))
        return dict(op=op, M=M, H=H, V=V, x_fmt=rng.choice(["e4m3", "e4m3", "e2m1"]),
                    w_fmt=rng.choice(["e2m1", "e2m1", "e4m3"]), dtype=dtype)
    V = _log_int(rng, 1000, 262144)
    return dict(op=op, N=_log_int(rng, 1, max(1, min(2048, 256 * 128256 // V // 2))), V=V,
                dtype=dtype, mode=rng.choice(["filters", "mixed", "temperature"]),
                sigma=round(rng.uniform(1.5, 5.0), 2))


# ---- inputs -------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _hidden(g, M, H, dtype):
    """Hidden states: normal, a few channels an order larger, as trained models have."""
    ch = torch.ones(H, device="cuda")
    ch[torch.randint(0, H, (max(1, H // 256),), generator=g, device="cuda")] = 12.0
    return (torch.randn((M, H), generator=g, device="cuda") * ch).to(dtype)


def _pow2(e):
    """2^e in FP32 from its bits, for integers e (clamped to the normal range)."""
    return ((e.to(torch.int32).clamp(-126, 127) + 127) << 23).view(torch.float32)


def _mx_bytes(v, fmt):
    """FP32 (rows, K) -> stored bytes and scale bytes."""
    bits, emin, vmax = FORMATS[fmt]
    rows, K = v.shape
    b = v.view(rows, K // BLOCK, BLOCK)
    e = _scale_exponent(b, fmt)
    x = (b * _pow2(-e)).view(rows, K)
    g = _to_grid(x, fmt).abs()
    _, ge = torch.frexp(g)
    ge = torch.clamp(ge - 1, min=emin)
    m = (g * _pow2(bits - ge)).to(torch.int32)  # in units of the last place
    code = torch.where(m >= (1 << bits), ((ge - emin) << bits) + m, m)
    code = (code | ((x < 0).to(torch.int32) << (3 if fmt == "e2m1" else 7))).to(torch.uint8)
    if fmt == "e2m1":
        code = code[:, 0::2] | (code[:, 1::2] << 4)
    return code.contiguous(), (e.view(rows, K // BLOCK) + 127).to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    st = dict(case=case)
    if op.startswith("rms"):
        M, H = case["M"], case["H"]
        st["x"] = _hidden(g, M, H, dt)
        st["res"] = _hidden(g, M, H, dt) if case["residual"] else None
        st["w"] = (torch.randn(H, generator=g, device="cuda") * 0.1 + 1.0 - case["offset"]).to(dt)
        if op == "rms_bwd":
            h = st["x"].float()
            st["rstd"] = torch.rsqrt((h * h).mean(1) + 1e-6)
            st["dy"] = _randn(g, (M, H), dt, 0.01)
            st["dh"] = _randn(g, (M, H), dt, 0.01) if case["residual"] else None
            if own:
                import vocabulary_cross_entropy_amd as vce
                st["ws"] = vce.rms_backward_workspace(M, H)
    elif op == "mx_round":
        st["x"] = _hidden(g, case["rows"], case["H"], dt)
    elif op == "mx_logits":
        M, H, V = case["M"], case["H"], case["V"]
        st["xq"], st["xs"] = _mx_bytes(_hidden(g, M, H, torch.float32), case["x_fmt"])
        W = torch.randn((V, H), generator=g, device="cuda") / math.sqrt(H)
        st["wq"], st["wsc"] = _mx_bytes(W, case["w_fmt"])
    else:
        N, V = case["N"], case["V"]
        z = torch.randn((N, V), generator=g, device="cuda") * case["sigma"]
        # a few likely continuations in every row
        top = torch.randint(0, V, (N, 8), generator=g, device="cuda")
        z.scatter_(1, top, torch.randn((N, 8), generator=g, device="cuda") * 2 +
                   3.5 * case["sigma"])
        st["z"] = z.to(dt)
        st["u"] = torch.rand(N, generator=g, device="cuda")

        def pick(vals, dtype=torch.float32):
            t = torch.tensor(vals, dtype=dtype, device="cuda")
            return t[torch.randint(0, len(vals), (N,), generator=g, device="cuda")]
        st["T"] = pick([0.6, 0.8, 1.0, 1.2])
        st["k"] = st["p"] = st["mp"] = None
        if case["mode"] == "filters":
            st["k"] = pick([20, 50, 200], torch.int32)
            st["p"] = pick([0.8, 0.9, 0.95])
            st["mp"] = pick([0.01, 0.05])
        elif case["mode"] == "mixed":
            st["T"] = pick([0.0, 0.7, 1.0, 1.0, 1.3])
            st["k"] = pick([0, 0, 1, 40, 1000], torch.int32)
            st["p"] = pick([1.0, 0.5, 0.9, 0.99])
            st["mp"] = pick([0.0, 0.0, 0.02, 0.1])
        if own:
            import vocabulary_cross_entropy_amd as vce
            st["ws"] = vce.ce_sample_workspace(N, V)
    return st


# ---- plain forms -------------------------------------------------------------------

def _scale_exponent(b, fmt):
    """Exponent of the least power of two s with amax <= vmax s, for blocks (..., 32)."""
    vmax = FORMATS[fmt][2]
    mv, ev = math.frexp(vmax)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = e - ev + (m > mv).to(e.dtype)
    return torch.clamp(torch.where(m == 0, torch.full_like(e, -127), e), -127, 127)


def _to_grid(v, fmt):
    bits, emin, vmax = FORMATS[fmt]
    _, e = torch.frexp(v)
    e = torch.clamp(e - 1, min=emin) - bits
    return torch.clamp(torch.round(v * _pow2(-e)) * _pow2(e), -vmax, vmax)


def _mx_values(v, fmt):
    rows, K = v.shape
    b = v.view(rows, K // BLOCK, BLOCK)
    e = _scale_exponent(b, fmt)
    return (_to_grid(b * _pow2(-e), fmt) * _pow2(e)).view(rows, K)


def _decode(q, s, fmt):
    bits, emin, _ = FORMATS[fmt]
    codes = 16 if fmt == "e2m1" else 256
    mag = torch.arange(codes // 2, device=q.device)
    ex, man = mag >> bits, mag & ((1 << bits) - 1)
    val = torch.where(ex > 0, (man + (1 << bits)).float() * _pow2(ex - 1 + emin - bits),
                      man.float() * 2.0 ** (emin - bits))
    table = torch.cat([val, -val])
    if fmt == "e2m1":
        q = torch.stack([q & 15, q >> 4], -1).view(q.shape[0], -1)
    rows, K = q.shape
    v = table[q.int()].view(rows, K // BLOCK, BLOCK)
    return (v * _pow2(s.int().unsqueeze(-1) - 127)).view(rows, K)


def _rms_plain(st, op):
    c = st["case"]
    w = st["w"].float() + c["offset"]
    x = st["x"].float()
    dt = DTYPES[c["dtype"]]
    if op == "rms_bwd":
        r = st["rstd"].unsqueeze(1)
        dy = st["dy"].float()
        gg = dy * w
        xh = x * r
        dx = r * (gg - xh * (gg * xh).mean(1, keepdim=True))
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        return [dx.to(dt), (dy * xh).sum(0)]
    h = x if st["res"] is None else x + st["res"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6)
    y = h * r * w
    out = [_mx_values(y, "e4m3").to(torch.bfloat16) if op == "rms_mx8" else y.to(dt), r.view(-1)]
    return out if st["res"] is None else out + [h.to(dt)]


def _sample_plain(st):
    z = st["z"].double()
    N, V = z.shape
    T = st["T"].double().unsqueeze(1)
    m = z.amax(1, keepdim=True)
    w = torch.exp((z - m) / torch.where(T == 0, torch.ones_like(T), T))
    ws, order = torch.sort(z, dim=1, descending=True, stable=True)
    ws = torch.gather(w, 1, order)
    keep = torch.ones_like(ws, dtype=torch.bool)
    rank = torch.arange(V, device=z.device).unsqueeze(0)
    if st["k"] is not None:
        k = st["k"].long().unsqueeze(1)
        keep &= (rank < k) | (k <= 0)
    if st["p"] is not None:
        p = st["p"].double().unsqueeze(1)
        wk = ws * keep
        cum = torch.cumsum(wk, 1)
        # kept while the mass before it has not reached p of the total
        keep &= (cum - wk < p * cum[:, -1:]) | (p >= 1) | (rank == 0)
    if st["mp"] is not None:
        keep &= ws >= st["mp"].double().unsqueeze(1)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    w = w * kept
    cum = torch.cumsum(w, 1)
    tot = cum[:, -1:]
    token = ((cum > st["u"].double().unsqueeze(1) * tot) & kept).int().argmax(1)
    logp = torch.log(torch.gather(w, 1, token.unsqueeze(1)) / tot)
    greedy = T.view(-1) == 0
    token = torch.where(greedy, (z == m).int().argmax(1), token)
    logp = torch.where(greedy, torch.zeros_like(logp.view(-1)), logp.view(-1))
    return [token, logp.float()]


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op.startswith("rms"):
        return _rms_plain(st, op)
    if op == "mx_round":
        return [_mx_values(st["x"].float(), c["fmt"]).to(torch.bfloat16)]
    if op == "mx_logits":
        x = _decode(st["xq"], st["xs"], c["x_fmt"])
        w = _decode(st["wq"], st["wsc"], c["w_fmt"])
        return [(x @ w.t()).to(DTYPES[c["dtype"]])]
    return _sample_plain(st)


def _run_own(st):
    import vocabulary_cross_entropy_amd as vce
    c = st["case"]
    op = c["op"]
    if op == "rms_bwd":
        return list(vce.rms_backward(st["dy"], st["x"], st["w"], st["rstd"], st["dh"],
                                     weight_offset=c["offset"], workspace=st["ws"]))
    if op == "rms_fwd":
        out = vce.rms_forward(st["x"], st["w"], st["res"], 1e-6, weight_offset=c["offset"])
        return [t for t in out if t is not None]
    if op == "rms_mx8":
        q, s, rstd, h = vce.rms_forward_mx8(st["x"], st["w"], st["res"], 1e-6,
                                            weight_offset=c["offset"])
        out = [vce.mx_dequantize(q, s, "e4m3"), rstd]
        return out if h is None else out + [h]
    if op == "mx_round":
        q, s = vce.mx_quantize(st["x"], c["fmt"])
        return [vce.mx_dequantize(q, s, c["fmt"])]
    if op == "mx_logits":
        return [vce.mx_logits(st["xq"], st["xs"], st["wq"], st["wsc"], x_fmt=c["x_fmt"],
                              w_fmt=c["w_fmt"], dtype=DTYPES[c["dtype"]])]
    return list(vce.ce_sample(st["z"], st["u"], st["T"], st["k"], st["p"], st["mp"],
                              with_logprob=True, workspace=st["ws"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definitions in 64 bits ------------------------------------------------------

def _exact_mx(v, fmt):
    """Nearest representable value by enumeration of the format's positive grid."""
    bits, emin, vmax = FORMATS[fmt]
    pts = [k * 2.0 ** (emin - bits) for k in range(1 << bits)]
    e = emin
    while True:
        pts += [(1 + k / (1 << bits)) * 2.0 ** e for k in range(1 << bits)]
        if pts[-1] >= vmax:
            break
        e += 1
    grid = torch.tensor([p for p in pts if p <= vmax], dtype=torch.float64, device=v.device)
    mid = (grid[1:] + grid[:-1]) / 2
    b = v.view(v.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.exp2(torch.ceil(torch.log2(amax / vmax)))
    s = torch.where(s * vmax < amax, s * 2, s)
    s = torch.where(s * vmax / 2 >= amax, s / 2, s)
    s = torch.clamp(s, min=2.0 ** -127)
    a = (b.abs() / s).contiguous()
    # ties go to the even mantissa: grid positions alternate, even ones are even
    lo = torch.searchsorted(mid, a, right=False)
    hi = torch.searchsorted(mid, a, right=True)
    idx = torch.where(lo % 2 == 0, lo, hi)
    return (torch.sign(b) * grid[idx] * s).view(v.shape)


def _exact_decode(q, s, fmt):
    if fmt == "e2m1":
        q = torch.stack([q & 15, q >> 4], -1).view(q.shape[0], -1).short()
        sign, ex, man, bias, mb = q >> 3, (q >> 1) & 3, q & 1, 1, 1
    else:
        q = q.short()
        sign, ex, man, bias, mb = q >> 7, (q >> 3) & 15, q & 7, 7, 3
    frac = man.double() / (1 << mb) + (ex > 0)
    v = frac * torch.exp2((torch.clamp(ex, min=1) - bias).double())
    v = torch.where(sign > 0, -v, v)
    sc = torch.exp2(s.double() - 127).repeat_interleave(BLOCK, dim=1)
    return v * sc


def _exact_sample(st):
    z = st["z"].float().cpu().numpy().astype(np.float64)
    N, V = z.shape

    def host(name, off):
        t = st[name]
        return np.full(N, off) if t is None else t.cpu().numpy().astype(np.float64)
    u, T, k, p, mp = (host("u", 0), host("T", 1.0), host("k", 0), host("p", 1.0),
                      host("mp", 0.0))
    tok = np.zeros(N, np.int64)
    lp = np.zeros(N, np.float64)
    for r in range(N):
        if T[r] == 0:
            tok[r] = int(np.argmax(z[r]))
            continue
        w = np.exp((z[r] - z[r].max()) / T[r])
        sel = np.arange(V)
        if (0 < k[r] < V) or p[r] < 1:
            sel = np.argsort(-z[r], kind="stable")
            if 0 < k[r] < V:
                sel = sel[:int(k[r])]
            if p[r] < 1:
                cum = np.cumsum(w[sel])
                sel = sel[:int(np.searchsorted(cum, p[r] * cum[-1], side="left")) + 1]
        sel = np.sort(sel[w[sel] >= mp[r]])
        cum = np.cumsum(w[sel])
        j = min(int(np.searchsorted(cum, u[r] * cum[-1], side="right")), len(sel) - 1)
        tok[r] = sel[j]
        lp[r] = math.log(w[sel[j]] / cum[-1])
    return [torch.from_numpy(tok), torch.from_numpy(lp)]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "sample":
        return _exact_sample(st)
    if op == "mx_round":
        return [_exact_mx(st["x"].double(), case["fmt"])]
    if op == "mx_logits":
        x = _exact_decode(st["xq"], st["xs"], case["x_fmt"])
        return [x @ _exact_decode(st["wq"], st["wsc"], case["w_fmt"]).t()]
    x, w = st["x"].double(), st["w"].double() + case["offset"]
    if op == "rms_bwd":
        r = st["rstd"].double().unsqueeze(1)
        dy = st["dy"].double()
        H = case["H"]
        # dx_j = r w_j dy_j - r^3 x_j / H sum_i w_i dy_i x_i
        dot = (dy * w * x).sum(1, keepdim=True)
        dx = r * w * dy - r ** 3 * x * dot / H
        if st["dh"] is not None:
            dx = dx + st["dh"].double()
        return [dx, (dy * x * r).sum(0)]
    h = x if st["res"] is None else x + st["res"].double()
    r = 1.0 / torch.sqrt((h ** 2).sum(1) / case["H"] + 1e-6)
    y = h * w * r.unsqueeze(1)
    out = [_exact_mx(y, "e4m3") if op == "rms_mx8" else y, r]
    return out if st["res"] is None else out + [h]


def work(case):
    op = case["op"]
    es = ELEM[case["dtype"]]
    if op.startswith("rms"):
        n = case["M"] * case["H"]
        if op == "rms_bwd":
            return dict(bytes=n * es * (4 if case["residual"] else 3) + case["H"] * (es + 4) +
                        case["M"] * 4, flops=10 * n)
        out = 2 if op == "rms_mx8" else es
        return dict(bytes=n * es * (3 if case["residual"] else 1) + n * out + case["H"] * es +
                    case["M"] * 4, flops=5 * n)
    if op == "mx_round":
        n = case["rows"] * case["H"]
        return dict(bytes=n * (es + 2), flops=4 * n)
    if op == "mx_logits":
        M, H, V = case["M"], case["H"], case["V"]
        size = {"e4m3": 1 + 1 / 32, "e2m1": 0.5 + 1 / 32}
        return dict(bytes=int(M * H * size[case["x_fmt"]] + V * H * size[case["w_fmt"]]) +
                    M * V * es, flops=2 * M * H * V)
    n = case["N"] * case["V"]
    return dict(bytes=n * es + case["N"] * 32, flops=4 * n)
