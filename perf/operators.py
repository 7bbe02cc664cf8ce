"""The workloads that the adapters of many requests and the distillation loss are measured on.

Four operators: the linear layer over a shared 4-bit base weight in which every token uses the
low-rank adapter of its own request (forward and backward), and the distillation loss from a
teacher's top logits (forward and backward).  Each case is computed either in a plain form of
elementary torch operations in fp32 (`own` false) or by this package's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step of four requests, each its own adapter: latency counts
        dict(name="fwd_tokens4", op="fwd", M=4, N=4096, K=4096, n=4, r=16, dt="bf16", dq=True, rows="tokens"),
        # a decode batch of 48 requests over 32 adapters, some requests without one
        dict(name="fwd_tokens48", op="fwd", M=48, N=8192, K=8192, n=32, r=16, dt="bf16", dq=True, rows="tokens"),
        # drafted or chunked tokens of a few requests on the widest projection, fp16, single-level constants
        dict(name="fwd_tokens112_fp16", op="fwd", M=112, N=28672, K=8192, n=6, r=64, dt="fp16", dq=False, rows="prompts"),
        # prompts and single tokens in one batch, a ragged number of tokens
        dict(name="fwd_mixed777", op="fwd", M=777, N=11008, K=4096, n=24, r=32, dt="bf16", dq=True, rows="mixed"),
        # a large batch of prompts
        dict(name="fwd_prompts4096", op="fwd", M=4096, N=22016, K=8192, n=12, r=64, dt="bf16", dq=True, rows="prompts"),
        # the backward of a small layer and batch: many small kernels
        dict(name="bwd_100", op="bwd", M=100, N=1000, K=1024, n=3, r=8, dt="bf16", dq=True, rows="prompts"),
        # fp16 training of six adapters, one token short of full tiles
        dict(name="bwd_2047_fp16", op="bwd", M=2047, N=4096, K=11008, n=6, r=16, dt="fp16", dq=True, rows="prompts"),
        # forward and backward of a training step over eight adapters
        dict(name="step_2048", op="step", M=2048, N=8192, K=8192, n=8, r=64, dt="bf16", dq=True, rows="prompts"),
        # the loss of a few rows over a long vocabulary of odd length: latency counts
        dict(name="distill_fwd_5", op="distill_fwd", M=5, V=50001, k=20, dt="bf16", out="bf16", T=1.0),
        # the loss of a full batch over a long vocabulary
        dict(name="distill_fwd_4096", op="distill_fwd", M=4096, V=128000, k=64, dt="bf16", out="bf16", T=2.0),
        # the gradient from fp32 logits of odd length, rounded to the dtype that the layer's backward takes
        dict(name="distill_bwd_1023", op="distill_bwd", M=1023, V=50001, k=100, dt="fp32", out="bf16", T=1.5),
        # loss and gradient as a training step calls them
        dict(name="distill_step_4096", op="distill_step", M=4096, V=32000, k=32, dt="bf16", out="bf16", T=2.0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "step", "distill_fwd", "distill_bwd", "distill_step"])
    if op.startswith("distill"):
        c = dict(op=op, M=_spread(rng, 1, 4096), V=_spread(rng, 1000, 128000), k=_spread(rng, 1, 256),
                 dt=rng.choice(["bf16", "fp16", "fp32"]), T=rng.choice([0.7, 1.0, 2.0, 4.0]))
        c["out"] = "bf16" if c["dt"] == "fp32" and rng.random() < 0.5 else c["dt"]
        c["M"] = max(1, min(c["M"], 250_000_000 // c["V"] // (2 if op == "distill_step" else 1)))
        return c
    N, K = _spread(rng, 256, 28672), 64 * _spread(rng, 4, 172)
    if rng.random() < 0.7:
        N = max(8, N // 8 * 8)
    M = _spread(rng, 1, 4096)
    M = max(1, min(M, 700_000_000_000 // (2 * N * K) // (1 if op == "fwd" else 3)))
    n = _spread(rng, 1, 32)
    r = rng.choice([4, 8, 16, 24, 32, 64, 128])
    n = max(1, min(n, 2048 // r))
    return dict(op=op, M=M, N=N, K=K, n=n, r=r, dt=rng.choice(["bf16", "bf16", "fp16"]), dq=rng.random() < 0.75,
                rows=rng.choice(["tokens", "prompts", "mixed"]))


# ---------------------------------------------------------------------------- inputs


def _codebook():
    """The 16 NormalFloat values: 8 positive and 7 negative normal quantiles and zero, over the largest."""
    delta = ((1 - 1 / 30) + (1 - 1 / 32)) / 2
    pos = torch.special.ndtri(torch.linspace(delta, 0.5, 9, dtype=torch.float64)[:8])
    neg = -torch.special.ndtri(torch.linspace(delta, 0.5, 8, dtype=torch.float64)[:7])
    v = torch.cat([pos, neg, torch.zeros(1, dtype=torch.float64)]).sort().values
    return v / v.max()


def _requests(case, g):
    """Adapter of each token: requests of contiguous tokens (one token each for "tokens"), about one in eight without."""
    M, n = case["M"], case["n"]
    if case["rows"] == "tokens":
        lens = np.ones(M, np.int64)
    else:
        singles = M // 4 if case["rows"] == "mixed" else 0
        parts = max(1, min(n, M - singles))
        share = np.sort(g.integers(0, M - singles + 1, parts - 1))
        lens = np.concatenate([np.diff(np.concatenate([[0], share, [M - singles]])), np.ones(singles, np.int64)])
    ids = np.concatenate([g.permutation(n) for _ in range(-(-len(lens) // n))])[:len(lens)].astype(np.int32)
    if len(lens) > 1:
        ids[g.random(len(lens)) < 0.125] = -1
    return np.repeat(ids, lens)


def _linear_inputs(case, seed):
    M, N, K, n, r = case["M"], case["N"], case["K"], case["n"], case["r"]
    dt = DTYPES[case["dt"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    book = _codebook().cuda()
    edges = ((book[1:] + book[:-1]) / 2).float()
    x = torch.randn(N * K, generator=g, device="cuda").mul_(0.36)
    idx = torch.bucketize(x, edges, out_int32=True).to(torch.uint8)
    del x
    nb1 = N * K // 64
    s = dict(case=case, codes=(idx[0::2] << 4) | idx[1::2], book=book.float())
    if case["dq"]:
        s["c1_codes"] = torch.randn(nb1, generator=g, device="cuda").mul_(120).clamp_(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
        s["c2"] = torch.rand(-(-nb1 // 256), generator=g, device="cuda").mul_(2e-5).add_(2e-5)
        s["mu"] = torch.full((1,), 0.055, device="cuda")
    else:
        s["c1"] = torch.rand(nb1, generator=g, device="cuda").mul_(0.03).add_(0.04)

    def normal(shape, std):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dt)

    s["X"] = normal((M, K), 1.0)
    s["A"] = normal((n, r, K), K ** -0.5)
    s["B"] = normal((n, N, r), 0.05)
    s["idx"] = torch.from_numpy(_requests(case, np.random.default_rng(seed))).cuda()
    s["scales"] = torch.rand(n, generator=g, device="cuda").add_(0.5)
    if case["op"] != "fwd":
        s["dY"] = normal((M, N), 1.0 / 16)
    if case["op"] == "bwd":   # what the forward of the step has kept
        s["U"] = (_adapter_columns(s["X"].double() @ s["A"].double().reshape(n * r, K).t(), s["idx"], n, r)
                  .reshape(M, n, r).sum(1).float())
    return s


def _distill_inputs(case, seed):
    M, V, k = case["M"], case["V"], min(case["k"], case["V"])
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.randn(M, V, generator=g, device="cuda").mul_(2.5)
    # the teacher's answers: near the student's own, its k largest kept, some rows shorter, some without any
    few = min(M, max(1, 400_000_000 // V))
    t = torch.empty(M, k, device="cuda")
    idx = torch.empty(M, k, dtype=torch.int32, device="cuda")
    for m in range(0, M, few):
        v, i = torch.topk(z[m:m + few] + torch.randn(z[m:m + few].shape, generator=g, device="cuda"), k)
        t[m:m + few], idx[m:m + few] = v, i.int()
    have = torch.randint(k // 2, k + 1, (M, 1), generator=g, device="cuda").clamp_(min=1)
    have[torch.rand(M, 1, generator=g, device="cuda") < (0.1 if M > 1 else 0.0)] = 0
    idx[torch.arange(k, device="cuda")[None, :] >= have] = -1
    s = dict(case=case, logits=z.to(DTYPES[case["dt"]]), idx=idx, t=t, dloss=torch.full((M,), 1.0 / M, device="cuda"))
    if case["op"] == "distill_bwd":   # what the forward has kept
        s["lse"] = torch.logsumexp(s["logits"].double() / case["T"], 1).float()
    return s


def prepare(case, seed):
    s = _distill_inputs(case, seed) if case["op"].startswith("distill") else _linear_inputs(case, seed)
    if own:
        import bit_nf4_quantized_23_b200 as q4
        s["q4"] = q4
        if "codes" in s:   # the handle of the stored weight: the same buffers
            s["w"] = q4.NF4Weight(s["codes"], s.get("c1_codes"), s.get("c2"), s.get("mu"), case["N"], case["K"], "nf4",
                                  s.get("c1"), DTYPES[case["dt"]])
    return s


# ---------------------------------------------------------------------------- plain forms


def _adapter_columns(v, idx, n, r):
    """v [M, n*r] with the columns of every adapter but the row's own set to zero."""
    mine = idx[:, None] == torch.arange(n, device=idx.device, dtype=idx.dtype)[None, :]
    return torch.where(mine[:, :, None].expand(-1, -1, r).reshape(v.shape), v, torch.zeros((), dtype=v.dtype, device=v.device))


def _w_hat(s):
    c = s["case"]
    q = s["book"][torch.stack([s["codes"] >> 4, s["codes"] & 15], 1).reshape(-1, 64).int()]
    if c["dq"]:
        v8 = s["c1_codes"].view(torch.float8_e4m3fn).float()
        c1 = v8 * s["c2"].repeat_interleave(256)[:v8.numel()] + s["mu"]
    else:
        c1 = s["c1"]
    return (q * c1[:, None]).reshape(c["N"], c["K"]).to(DTYPES[c["dt"]]).float()


def _plain_fwd(s, Wh):
    c, dt = s["case"], DTYPES[s["case"]["dt"]]
    n, r = c["n"], c["r"]
    X = s["X"].float()
    U = _adapter_columns(X @ s["A"].float().reshape(n * r, -1).t(), s["idx"], n, r)
    sU = U * s["scales"].repeat_interleave(r)[None, :]
    Y = X @ Wh.t() + sU @ s["B"].float().transpose(1, 2).reshape(n * r, -1)
    return Y.to(dt), U.reshape(-1, n, r).sum(1)


def _plain_bwd(s, Wh, U):
    c, dt = s["case"], DTYPES[s["case"]["dt"]]
    n, r = c["n"], c["r"]
    X, dY = s["X"].float(), s["dY"].float()
    A, B = s["A"].float().reshape(n * r, -1), s["B"].float().transpose(1, 2).reshape(n * r, -1)
    scale = s["scales"].repeat_interleave(r)[None, :]
    dU = _adapter_columns(dY @ B.t(), s["idx"], n, r) * scale
    dX = dY @ Wh + dU @ A
    dA = dU.t() @ X
    sU = _adapter_columns(U.repeat(1, n), s["idx"], n, r) * scale
    dB = sU.t() @ dY
    return dX.to(dt), dA.reshape(n, r, -1), dB.reshape(n, r, -1).transpose(1, 2).contiguous()


def _teacher(s):
    """(p, log p) of each row's valid entries, zeros elsewhere, and the rows that have any."""
    valid = s["idx"] >= 0
    some = valid.any(1)
    t = torch.where(valid, s["t"] / s["case"]["T"], torch.full_like(s["t"], -torch.inf))
    t = torch.where(some[:, None], t, torch.zeros_like(t))
    t = t - t.max(1, keepdim=True).values
    logp = t - t.exp().sum(1, keepdim=True).log()
    p = torch.where(valid, logp.exp(), torch.zeros_like(t))
    return p, torch.where(valid, logp, torch.zeros_like(t)), some


def _plain_distill_fwd(s):
    T = s["case"]["T"]
    z = s["logits"].float() / T
    top = z.max(1, keepdim=True).values
    lse = (z - top).exp().sum(1).log() + top[:, 0]
    p, logp, some = _teacher(s)
    logq = z.gather(1, s["idx"].clamp(min=0).long()) - lse[:, None]
    return T * T * (p * (logp - logq)).sum(1), lse


def _plain_distill_bwd(s, lse):
    T = s["case"]["T"]
    p, _, some = _teacher(s)
    q = (s["logits"].float() / T - lse[:, None]).exp()
    g = q.scatter_add(1, s["idx"].clamp(min=0).long(), -p)
    g = g * torch.where(some, T * s["dloss"], torch.zeros_like(lse))[:, None]
    return g.to(DTYPES[s["case"]["out"]])


# ---------------------------------------------------------------------------- one pass


def run(s):
    c = s["case"]
    if own:
        q4, T = s["q4"], c.get("T")
        if c["op"] == "fwd":
            return q4.qlora_linear_fwd_adapters(s["w"], s["X"], s["A"], s["B"], s["idx"], s["scales"], save_U=False)[0]
        if c["op"] == "bwd":
            return q4.qlora_linear_bwd_adapters(s["w"], s["X"], s["dY"], s["A"], s["B"], s["idx"], s["scales"],
                                                U_saved=s["U"])
        if c["op"] == "step":
            Y, U = q4.qlora_linear_fwd_adapters(s["w"], s["X"], s["A"], s["B"], s["idx"], s["scales"])
            return (Y,) + q4.qlora_linear_bwd_adapters(s["w"], s["X"], s["dY"], s["A"], s["B"], s["idx"], s["scales"],
                                                       U_saved=U)
        if c["op"] == "distill_fwd":
            return q4.qlora_distill_topk_fwd(s["logits"], s["idx"], s["t"], T)
        if c["op"] == "distill_bwd":
            return q4.qlora_distill_topk_bwd(s["logits"], s["idx"], s["t"], s["lse"], s["dloss"], T,
                                             d_dtype=DTYPES[c["out"]])
        loss, lse = q4.qlora_distill_topk_fwd(s["logits"], s["idx"], s["t"], T)
        return loss, q4.qlora_distill_topk_bwd(s["logits"], s["idx"], s["t"], lse, s["dloss"], T,
                                               d_dtype=DTYPES[c["out"]])
    if c["op"] == "fwd":
        return _plain_fwd(s, _w_hat(s))[0]
    if c["op"] == "bwd":
        return _plain_bwd(s, _w_hat(s), s["U"])
    if c["op"] == "step":
        Wh = _w_hat(s)
        Y, U = _plain_fwd(s, Wh)
        return (Y,) + _plain_bwd(s, Wh, U)
    if c["op"] == "distill_fwd":
        return _plain_distill_fwd(s)
    if c["op"] == "distill_bwd":
        return _plain_distill_bwd(s, s["lse"])
    loss, lse = _plain_distill_fwd(s)
    return loss, _plain_distill_bwd(s, lse)


def work(case):
    """Each input read once and each output written once; products count two operations a multiply-add."""
    bytes_of = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"].startswith("distill"):
        M, V, k = case["M"], case["V"], min(case["k"], case["V"])
        b, o = bytes_of[case["dt"]], bytes_of[case["out"]]
        fwd, bwd = case["op"] != "distill_bwd", case["op"] != "distill_fwd"
        return {"bytes": M * V * (b + (o if bwd else 0)) + 8 * M * k + 8 * M, "flops": M * V * 3 * (fwd + bwd)}
    M, N, K, n, r = case["M"], case["N"], case["K"], case["n"], case["r"]
    fwd, bwd = case["op"] != "bwd", case["op"] != "fwd"
    used = min(n, M)
    nb1 = N * K // 64
    stored = N * K // 2 + (nb1 + nb1 // 64 if case["dq"] else 4 * nb1)
    b = stored + 2 * M * K + 2 * used * r * (N + K) + 4 * M + 4 * n
    f = 0
    if fwd:
        b += 2 * M * N
        f += 2 * M * N * K + 2 * M * r * (N + K)
    if bwd:
        b += 2 * M * N + 2 * M * K + 4 * n * r * (N + K) + (4 * M * r if not fwd else 0)
        f += 2 * M * N * K + 4 * M * r * (N + K)
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    if case["op"].startswith("distill"):
        s = _distill_inputs(case, seed)
        M, T = case["M"], case["T"]
        loss = torch.zeros(M, dtype=torch.float64, device="cuda")
        lse = torch.zeros(M, dtype=torch.float64, device="cuda")
        d = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda") if case["op"] != "distill_fwd" else None
        few = max(1, 200_000_000 // case["V"])
        for m in range(0, M, few):
            e = slice(m, min(M, m + few))
            logq = torch.log_softmax(s["logits"][e].double() / T, 1)
            lse[e] = torch.logsumexp(s["logits"][e].double() / T, 1)
            ok = s["idx"][e] >= 0
            any_row = ok.any(1)
            w = torch.softmax((s["t"][e].double() / T).masked_fill(~ok, -torch.inf), 1).nan_to_num(0.0).masked_fill(~ok, 0.0)
            at = s["idx"][e].long().clamp(min=0)
            loss[e] = T * T * (torch.special.xlogy(w, w) - w * logq.gather(1, at)).sum(1)
            if d is not None:
                # the kept lse is an fp32 input of the backward
                q = (s["logits"][e].double() / T - s["lse"][e].double()[:, None]).exp() if "lse" in s else logq.exp()
                d[e] = (q.scatter_add(1, at, -w) * T * s["dloss"][e].double()[:, None]).masked_fill(~any_row[:, None], 0.0)
        return (loss, lse) if case["op"] == "distill_fwd" else d if case["op"] == "distill_bwd" else (loss, d)
    s = _linear_inputs(case, seed)
    M, N, K, n, r = case["M"], case["N"], case["K"], case["n"], case["r"]
    hi, lo = torch.div(s["codes"], 16, rounding_mode="floor").long(), torch.remainder(s["codes"], 16).long()
    W = torch.empty(N * K // 2, 2, dtype=torch.float32, device="cuda")
    W[:, 0], W[:, 1] = s["book"][hi], s["book"][lo]
    del hi, lo
    c1 = s["c1"] if not case["dq"] else s["c1_codes"].view(torch.float8_e4m3fn).float()
    if case["dq"]:
        c1 = c1 * s["c2"][torch.arange(c1.numel(), device="cuda") // 256] + s["mu"]
    W = (W.reshape(-1, 64) * c1[:, None]).to(DTYPES[case["dt"]]).reshape(N, K).double()
    X, ids = s["X"].double(), s["idx"].tolist()
    groups = [(a, torch.tensor([m for m in range(M) if ids[m] == a], device="cuda", dtype=torch.long)) for a in range(n)]
    out = []
    U = torch.zeros(M, r, dtype=torch.float64, device="cuda")
    if case["op"] != "bwd":
        Y = X @ W.t()
        for a, rows in groups:
            U[rows] = X[rows] @ s["A"][a].double().t()
            Y[rows] += float(s["scales"][a]) * (U[rows] @ s["B"][a].double().t())
        if case["op"] == "fwd":
            return Y
        out.append(Y)
    else:
        U = s["U"].double()
    dY = s["dY"].double()
    dX = dY @ W
    dA = torch.zeros(n, r, K, dtype=torch.float64, device="cuda")
    dB = torch.zeros(n, N, r, dtype=torch.float64, device="cuda")
    for a, rows in groups:
        dU = float(s["scales"][a]) * (dY[rows] @ s["B"][a].double())
        dX[rows] += dU @ s["A"][a].double()
        dA[a] = dU.t() @ X[rows]
        dB[a] = float(s["scales"][a]) * (dY[rows].t() @ U[rows])
    return tuple(out + [dX, dA, dB])
