"""Cases of the layer operators that stand next to the gated delta rule, and their plain forms.

Three operators, each with the direction(s) a program runs:

  scan   the gated linear recurrence per channel, h_t = alpha_t h_{t-1} + beta_t x_t with
         log alpha = -exp(A_log) softplus(a + dt_bias) and beta = sigmoid(b): one token ("step"),
         whole sequences ("fwd"), and a training pass ("train": outputs and every gradient);
  ffn    both projections of a gated feed-forward block with the activation and the product,
         h = silu(x Wg^T) * (x Wu^T): "fwd", and "train" with the gradients of x, Wg and Wu;
  ce     softmax cross entropy of x W^T over a vocabulary, the loss of each token: "fwd", and
         "train" with the gradients of x and W.

With ``own`` false, ``run`` is the operator in elementary torch operations in 32 bits, rounded
once at the end; with ``own`` true it is the library's entry points.
"""
import math

import torch

own = False

# Sizes: 16 heads of 128 channels give the width 2048 and batches of 4 sequences of 4096 tokens
# are the library's training shape; 256 sequences of 32 heads of 128 its decode shape; the packed
# lengths are those of its packed workload. Vocabularies and hidden widths are generic.
PACKED = "6225,1640,5975,962,2975,6224,2034,4541"


def listed():
    return [
        # one token of one sequence: a serving loop's smallest call, latency only
        dict(name="scan_step_n1_d2048", op="scan", do="step", N=1, D=2048, dtype="bf16"),
        # one token for a full decode batch
        dict(name="scan_step_n256_d4096", op="scan", do="step", N=256, D=4096, dtype="bf16"),
        # a training pass over the usual batch
        dict(name="scan_train_b4_t4096_d2048", op="scan", do="train", lengths="4096,4096,4096,4096", packed=False, D=2048, dtype="bf16"),
        # prefill of one long document: few channels next to the length
        dict(name="scan_fwd_b1_t131072_d1024", op="scan", do="fwd", lengths="131072", packed=False, D=1024, dtype="bf16"),
        # packed documents of unequal lengths, one empty and one of a single token, in 32 bits
        dict(name="scan_train_packed_fp32", op="scan", do="train", lengths=PACKED + ",0,1", packed=True, D=520, dtype="fp32"),
        # the block for one token: its weights are read once for one row
        dict(name="ffn_fwd_m1", op="ffn", do="fwd", M=1, D=2048, F=8192, dtype="bf16"),
        # the block for a full decode batch
        dict(name="ffn_fwd_m256", op="ffn", do="fwd", M=256, D=2048, F=8192, dtype="bf16"),
        # a training pass over the usual batch
        dict(name="ffn_train_m16384", op="ffn", do="train", M=16384, D=2048, F=8192, dtype="bf16"),
        # a ragged batch and an odd hidden width, in 32 bits
        dict(name="ffn_train_odd_fp32", op="ffn", do="train", M=1021, D=1024, F=2731, dtype="fp32"),
        # scoring a few candidate tokens: the vocabulary's weights are read once
        dict(name="ce_fwd_n16_v65536", op="ce", do="fwd", N=16, D=2048, V=65536, dtype="bf16"),
        # a training pass over the usual batch with a large vocabulary
        dict(name="ce_train_n16384_v65536", op="ce", do="train", N=16384, D=2048, V=65536, dtype="bf16"),
        # a ragged batch and an odd vocabulary
        dict(name="ce_train_n1021_v32003", op="ce", do="train", N=1021, D=1024, V=32003, dtype="bf16"),
    ]


def _log_size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "ffn", "ce"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "scan":
        # widths: any, from a few channels up; a training pass stays within the usual batch's cost
        do = rng.choice(["step", "fwd", "train", "train"])
        D = _log_size(rng, 48, 4096)
        if rng.random() < 0.7:
            D = max(8, D // 8 * 8)
        if do == "step":
            return dict(op=op, do=do, N=_log_size(rng, 1, 512), D=D, dtype=dtype)
        most = (4 * 4096 * 2048 if do == "train" else 131072 * 1024) // D
        total = _log_size(rng, 16, max(17, min(131072, most)))
        packed = rng.random() < 0.5
        n = rng.randint(1, 9)
        if packed:
            at = sorted(rng.randint(0, total) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + at, at + [total])]
        else:
            lens = [max(1, total // n)] * n
        return dict(op=op, do=do, lengths=",".join(map(str, lens)), packed=packed, D=D, dtype=dtype)
    # model widths are multiples of 8; token counts, hidden widths and vocabularies are any number
    do = rng.choice(["fwd", "train", "train"])
    D = _log_size(rng, 256, 4096) // 8 * 8
    if op == "ffn":
        # the largest listed training pass: 16384 tokens, 2048 x 8192 (in 32 bits a fortieth of it)
        M, F = _log_size(rng, 1, 16384), _log_size(rng, 500, 11000)
        most = 16384 * 2048 * 8192 // (40 if dtype == "fp32" else 1)
        M = max(1, min(M, most // (D * F)))
        return dict(op=op, do=do, M=M, D=D, F=F, dtype=dtype)
    N, V = _log_size(rng, 1, 16384), _log_size(rng, 1000, 131000)
    most = 16384 * 2048 * 65536 // (80 if dtype == "fp32" else 1)
    N = max(1, min(N, most // (D * V)))
    return dict(op=op, do=do, N=N, D=D, V=V, dtype=dtype)


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case):
    return [int(s) for s in case["lengths"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, D = _dt(case), case["D"]

    def randn(*shape, std=1.0):
        t = torch.empty(shape, dtype=torch.float32, device="cuda")
        return t.normal_(0.0, std, generator=g)

    s = dict(case=case)
    if case["op"] == "scan":
        # the library's layer initialisation: rates U(1, 16) and time steps logU(0.001, 0.1) per
        # channel, so that channels remember from one to about a thousand tokens
        s["A_log"] = torch.empty(D, device="cuda").uniform_(1.0, 16.0, generator=g).log_()
        step = torch.empty(D, device="cuda").uniform_(math.log(1e-3), math.log(0.1), generator=g).exp_()
        s["dt_bias"] = torch.log(torch.expm1(step))
        if case["do"] == "step":
            N = case["N"]
            for k in ("x", "a", "b"):
                s[k] = randn(N, D).to(dt)
            s["state"] = randn(N, D)
            return s
        lens = _lens(case)
        B, T = (1, sum(lens)) if case["packed"] else (len(lens), lens[0])
        for k in ("x", "a", "b"):
            s[k] = randn(B, T, D).to(dt)
        s["h0"] = randn(len(lens), D)
        s["cu"] = None
        if case["packed"]:
            s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        if case["do"] == "train":
            s["dout"], s["dhT"] = randn(B, T, D).to(dt), randn(len(lens), D)
        return s
    if case["op"] == "ffn":
        M, F = case["M"], case["F"]
        s["x"] = randn(M, D).to(dt)
        s["wg"], s["wu"] = randn(F, D, std=D ** -0.5).to(dt), randn(F, D, std=D ** -0.5).to(dt)
        if case["do"] == "train":
            s["dh"] = randn(M, F).to(dt)
        return s
    N, V = case["N"], case["V"]
    s["x"], s["w"] = randn(N, D).to(dt), randn(V, D, std=2.0 * D ** -0.5).to(dt)
    t = torch.empty(N, device="cuda", dtype=torch.int64).random_(0, V, generator=g)
    # one token in ten is padding and bears no loss
    t[torch.empty(N, device="cuda").uniform_(0.0, 1.0, generator=g) < 0.1] = -100
    s["t"] = t
    if case["do"] == "train":
        ok = t >= 0
        s["dloss"] = ok.float() / ok.sum().clamp(min=1)  # the mean over the tokens that count
    return s


def run(state):
    do = state["case"]["do"]
    if own:
        return {"scan": _own_scan, "ffn": _own_ffn, "ce": _own_ce}[state["case"]["op"]](state, do)
    return {"scan": _plain_scan, "ffn": _plain_ffn, "ce": _plain_ce}[state["case"]["op"]](state, do)


# ------------------------------------------------------------------ the library's entry points


def _own_scan(s, do):
    from gated_delta_rule_70_amd import binding

    par = (s["x"], s["a"], s["b"], s["A_log"], s["dt_bias"])
    if do == "step":
        out, state = binding.channel_scan_step(*par, s["state"])
        return dict(out=out, state=state)
    out, hT, states = binding.channel_scan_fwd(*par, s["h0"], s["cu"], want_states=do == "train")
    if do == "fwd":
        return dict(out=out, hT=hT)
    dx, da, db, dA_log, ddt_bias, dh0 = binding.channel_scan_bwd(*par, states, s["dout"], s["cu"], s["dhT"])
    return dict(out=out, hT=hT, dx=dx, da=da, db=db, dA_log=dA_log, ddt_bias=ddt_bias, dh0=dh0)


def _own_ffn(s, do):
    from gated_delta_rule_70_amd import binding

    h, gate, up = binding.gated_ffn_fwd(s["x"], s["wg"], s["wu"], want_saved=do == "train")
    if do == "fwd":
        return dict(h=h)
    dx, dwg, dwu = binding.gated_ffn_bwd(s["x"], s["wg"], s["wu"], gate, up, s["dh"])
    return dict(h=h, dx=dx, dwg=dwg, dwu=dwu)


def _own_ce(s, do):
    from gated_delta_rule_70_amd import binding

    loss, lse = binding.linear_ce_fwd(s["x"], s["w"], s["t"])
    if do == "fwd":
        return dict(loss=loss, lse=lse)
    dx, dw = binding.linear_ce_bwd(s["x"], s["w"], s["t"], lse, s["dloss"])
    return dict(loss=loss, lse=lse, dx=dx, dw=dw)


# ------------------------------------------------------------------ the plain forms


def _gates(s):
    u = s["a"].float() + s["dt_bias"]
    rate = s["A_log"].exp()
    soft = u.clamp(min=0) + torch.log1p(torch.exp(-u.abs()))
    return u, -rate * soft, rate, torch.sigmoid(s["b"].float())


def _linear_scan(alpha, v):
    """h_t = alpha_t h_{t-1} + v_t along dim 1 from zero, by doubling: after a pass with distance
    d, (p_t, h_t) hold the map over the last 2d steps."""
    h, p, d, T = v, alpha, 1, v.shape[1]
    while d < T:
        h = torch.cat([h[:, :d], torch.addcmul(h[:, d:], p[:, d:], h[:, :-d])], 1)
        if 2 * d < T:
            p = torch.cat([p[:, :d], p[:, d:] * p[:, :-d]], 1)
        d *= 2
    return h


def _edges(s, T):
    """Which (row, token) begins and ends each sequence, and which sequences have tokens."""
    if s["cu"] is None:
        n = s["x"].shape[0]
        rows = torch.arange(n, device="cuda")
        zero = torch.zeros_like(rows)
        return rows, zero, rows, zero + (T - 1), torch.ones(n, dtype=torch.bool, device="cuda")
    cu = s["cu"].long()
    some = cu[1:] > cu[:-1]
    zero = torch.zeros_like(cu[1:])
    return zero, cu[:-1].clamp(max=T - 1), zero, (cu[1:] - 1).clamp(min=0), some


def _put_add(t, rows, cols, some, value):
    """t with value added at [rows, cols], for the sequences that have tokens."""
    return t.index_put((rows, cols), torch.where(some[:, None], value, torch.zeros_like(value)), accumulate=True)


def _plain_scan(s, do):
    dt = s["x"].dtype
    u, log_alpha, rate, beta = _gates(s)
    alpha, x = log_alpha.exp(), s["x"].float()
    v = beta * x
    if do == "step":
        h = alpha * s["state"] + v
        return dict(out=h.to(dt), state=h)
    T = x.shape[1]
    r0, t0, r1, t1, some = _edges(s, T)
    first = torch.zeros(x.shape[:2], device=x.device).index_put((r0, t0), some.float(), accumulate=True) > 0
    cut = torch.where(first[..., None], torch.zeros_like(alpha), alpha)  # no carry into a sequence
    a0 = alpha[r0, t0]
    h = _linear_scan(cut, _put_add(v, r0, t0, some, a0 * s["h0"]))
    hT = torch.where(some[:, None], h[r1, t1], s["h0"])
    if do == "fwd":
        return dict(out=h.to(dt), hT=hT)
    # dh_t = dout_t + alpha_{t+1} dh_{t+1}, within a sequence
    dv = _put_add(s["dout"].float(), r1, t1, some, s["dhT"])
    nxt = torch.cat([cut[:, 1:], torch.zeros_like(cut[:, :1])], 1)
    dh = _linear_scan(nxt.flip(1), dv.flip(1)).flip(1)
    prev = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    prev = _put_add(torch.where(first[..., None], torch.zeros_like(prev), prev), r0, t0, some, s["h0"])
    dlog = alpha * prev * dh
    da = -rate * torch.sigmoid(u) * dlog
    return dict(out=h.to(dt), hT=hT, dx=(beta * dh).to(dt), da=da.to(dt),
                db=(beta * (1 - beta) * x * dh).to(dt), dA_log=(dlog * log_alpha).sum((0, 1)),
                ddt_bias=da.sum((0, 1)), dh0=torch.where(some[:, None], a0 * dh[r0, t0], s["dhT"]))


def _plain_ffn(s, do):
    dt = s["x"].dtype
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    gate, up = x @ wg.T, x @ wu.T
    sig = torch.sigmoid(gate)
    act = gate * sig
    h = (act * up).to(dt)
    if do == "fwd":
        return dict(h=h)
    dh = s["dh"].float()
    dup = dh * act
    dgate = dh * up * (sig * (1 + gate * (1 - sig)))
    return dict(h=h, dx=(dgate @ wg + dup @ wu).to(dt), dwg=(dgate.T @ x).to(dt), dwu=(dup.T @ x).to(dt))


def _plain_ce(s, do):
    dt = s["x"].dtype
    x, w, t = s["x"].float(), s["w"].float(), s["t"]
    logits = x @ w.T
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    lse = (top + total.log())[:, 0]
    ok = t >= 0
    at = t.clamp(min=0)[:, None]
    loss = torch.where(ok, lse - logits.gather(1, at)[:, 0], torch.zeros_like(lse))
    if do == "fwd":
        return dict(loss=loss, lse=lse)
    scale = torch.where(ok, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    d = e * (scale / total)
    d.scatter_add_(1, at, -scale)
    return dict(loss=loss, lse=lse, dx=(d @ w).to(dt), dw=(d.T @ x).to(dt))


# ------------------------------------------------------------------ work and the exact values


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    D, do = case["D"], case["do"]
    if case["op"] == "scan":
        if do == "step":
            n = case["N"] * D
            return dict(bytes=n * (4 * es + 8) + 8 * D, flops=12 * n)
        lens = _lens(case)
        n, st = sum(lens) * D, 4 * len(lens) * D
        if do == "fwd":
            return dict(bytes=4 * n * es + 2 * st + 8 * D, flops=12 * n)
        # x, a, b, dout in; out, dx, da, db out; initial and final states with their gradients
        return dict(bytes=8 * n * es + 4 * st + 16 * D, flops=40 * n)
    if case["op"] == "ffn":
        M, F = case["M"], case["F"]
        if do == "fwd":
            return dict(bytes=es * (M * D + 2 * F * D + M * F), flops=4 * M * D * F)
        return dict(bytes=es * (2 * M * D + 4 * F * D + 2 * M * F), flops=12 * M * D * F)
    N, V = case["N"], case["V"]
    if do == "fwd":
        return dict(bytes=es * (N * D + V * D) + 16 * N, flops=2 * N * D * V)
    return dict(bytes=2 * es * (N * D + V * D) + 20 * N, flops=6 * N * D * V)


def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return {"scan": _exact_scan, "ffn": _exact_ffn, "ce": _exact_ce}[case["op"]](f, case)


def _exact_scan(s, case):
    do = case["do"]
    rate = s["A_log"].exp()
    u = s["a"] + s["dt_bias"]
    log_alpha = -rate * torch.nn.functional.softplus(u, threshold=200.0)
    alpha, beta = log_alpha.exp(), 1 / (1 + torch.exp(-s["b"]))
    if do == "step":
        h = alpha * s["state"] + beta * s["x"]
        return dict(out=h, state=h)
    lens = _lens(case)
    if sum(lens) > 300000:
        return None
    out, hT = torch.empty_like(s["x"]), torch.empty_like(s["h0"])
    dx, da, db, dlog = (torch.empty_like(s["x"]) for _ in range(4)) if do == "train" else (None,) * 4
    dh0 = torch.empty_like(hT)
    # the recurrence as written, token by token; equal lengths side by side
    spans = [(slice(0, None), slice(0, lens[0]), slice(0, None))]
    if case["packed"]:
        ends = [sum(lens[:i]) for i in range(len(lens) + 1)]
        spans = [(slice(0, 1), slice(ends[i], ends[i + 1]), slice(i, i + 1)) for i in range(len(lens))]
    for rows, toks, seqs in spans:
        al, v = alpha[rows, toks], beta[rows, toks] * s["x"][rows, toks]
        T = al.shape[1]
        h = s["h0"][seqs]
        prev = torch.empty_like(al)
        o = out[rows, toks]
        for t in range(T):
            prev[:, t] = h
            h = torch.addcmul(v[:, t], al[:, t], h)
            o[:, t] = h
        hT[seqs] = h
        if do != "train":
            continue
        g, up = s["dhT"][seqs], s["dout"][rows, toks]
        dh = torch.empty_like(al)
        for t in range(T - 1, -1, -1):
            g = g + up[:, t]
            dh[:, t] = g
            g = al[:, t] * g
        dh0[seqs] = g
        be, xx = beta[rows, toks], s["x"][rows, toks]
        dx[rows, toks] = be * dh
        db[rows, toks] = xx * dh * be * (1 - be)
        dlog[rows, toks] = dh * prev * al
        da[rows, toks] = -dlog[rows, toks] * rate / (1 + torch.exp(-u[rows, toks]))
    if do == "fwd":
        return dict(out=out, hT=hT)
    return dict(out=out, hT=hT, dx=dx, da=da, db=db, dA_log=(dlog * log_alpha).sum((0, 1)), ddt_bias=da.sum((0, 1)), dh0=dh0)


def _exact_ffn(s, case):
    x, wg, wu = s["x"], s["wg"], s["wu"]
    if case["M"] * case["D"] * case["F"] > 16384 * 2048 * 8192:
        return None
    gate, up = torch.nn.functional.linear(x, wg), torch.nn.functional.linear(x, wu)
    act = torch.nn.functional.silu(gate)
    h = act * up
    if case["do"] == "fwd":
        return dict(h=h)
    dup, dact = s["dh"] * act, s["dh"] * up
    sg = 1 / (1 + torch.exp(-gate))
    dgate = dact * (sg + gate * sg * (1 - sg))
    return dict(h=h, dx=torch.mm(dgate, wg) + torch.mm(dup, wu), dwg=torch.mm(dgate.T, x), dwu=torch.mm(dup.T, x))


def _exact_ce(s, case):
    x, w, t = s["x"], s["w"], s["t"]
    if case["N"] * case["D"] * case["V"] > 16384 * 2048 * 65536:
        return None
    logits = torch.nn.functional.linear(x, w)
    logp = torch.log_softmax(logits, 1)
    ok = t >= 0
    at = torch.where(ok, t, torch.zeros_like(t))[:, None]
    loss = torch.where(ok, -logp.gather(1, at)[:, 0], torch.zeros_like(logits[:, 0]))
    lse = torch.logsumexp(logits, 1)
    del logits
    if case["do"] == "fwd":
        return dict(loss=loss, lse=lse)
    d = logp.exp_()
    d.scatter_add_(1, at, -torch.ones_like(loss)[:, None])
    d *= torch.where(ok, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    return dict(loss=loss, lse=lse, dx=torch.mm(d, w), dw=torch.mm(d.T, x))
