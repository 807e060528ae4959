"""Measured cases of the routed-token and int8 operators.

Five operators, each in its plain form (elementary torch operations in 32 bits, 64 for the rounding
decisions of the quantiser) and as a caller of the library reaches it:

  dispatch  tokens sorted by expert: row maps, expert offsets and the gathered rows
  combine   the experts' rows back to their tokens, with the routing weights applied
  grad      the gradients of both: d(rows), d(weights) of combine and d(tokens) of dispatch
  i8        bf16 rows times an int8 matrix, one scale per row (taken on the fly) and per channel
  i8_moe    the same over experts: the fused gate+up with SiLU, or the down projection
"""
import math

import torch

own = False

BF16, F32 = "bf16", "fp32"
DT = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one decode step of 64 sequences over 512 experts, top-10: launch latency counts
        dict(name="dispatch decode", op="dispatch", T=64, k=10, E=512, H=2048, dtype=BF16, drop=False),
        # a prefill chunk of the same layer, padded tokens (no expert) among it
        dict(name="dispatch prefill", op="dispatch", T=2048, k=10, E=512, H=2048, dtype=BF16, drop=True),
        # few wide experts, a long chunk whose length is odd
        dict(name="dispatch long", op="dispatch", T=7235, k=2, E=8, H=5120, dtype=BF16, drop=False),
        # decode: the down projection's fp32 rows back to bf16 tokens
        dict(name="combine decode", op="combine", T=64, k=10, E=512, H=2048, dtype=F32, out=BF16, drop=False),
        # prefill chunk, bf16 rows
        dict(name="combine prefill", op="combine", T=2048, k=10, E=512, H=2048, dtype=BF16, out=BF16, drop=True),
        # odd sizes: a token count and a width that no vector divides, fp32
        dict(name="grad odd", op="grad", T=333, k=3, E=7, H=1001, dtype=F32, out=F32, drop=True),
        # a training step's micro-batch
        dict(name="grad train", op="grad", T=2048, k=10, E=512, H=2048, dtype=BF16, out=BF16, drop=False),
        # one token through the 27B gate or up matrix
        dict(name="i8 token", op="i8", M=1, N=17408, K=5120, out=BF16),
        # a decode batch through the 27B down matrix
        dict(name="i8 decode", op="i8", M=64, N=5120, K=17408, out=F32),
        # a prefill chunk through the 27B gate or up matrix
        dict(name="i8 prefill", op="i8", M=2048, N=17408, K=5120, out=BF16),
        # decode over 512 routed experts: fused gate+up
        dict(name="i8_moe decode", op="i8_moe", part="gate_up", T=64, k=10, E=512, N=512, K=2048, out=BF16),
        # prefill chunk over the same experts: down projection
        dict(name="i8_moe prefill", op="i8_moe", part="run", T=2048, k=10, E=512, N=2048, K=512, out=F32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "grad", "i8", "i8", "i8_moe"])
    if op in ("dispatch", "combine", "grad"):
        E = _log(rng, 2, 512)
        k = min(E, rng.randint(1, 10))
        T = _log(rng, 1, 4096)
        H = rng.choice([_log(rng, 16, 5120), 8 * _log(rng, 2, 640)])
        c = dict(op=op, T=T, k=k, E=E, H=H, dtype=rng.choice([BF16, F32]), drop=rng.random() < 0.5)
        if op != "dispatch":
            c["out"] = rng.choice([BF16, F32])
        return c
    if op == "i8":
        return dict(op=op, M=_log(rng, 1, 2048), N=_log(rng, 64, 17408), K=16 * _log(rng, 4, 320), out=rng.choice([BF16, F32]))
    E = _log(rng, 2, 256)
    part = rng.choice(["gate_up", "run"])
    return dict(op=op, part=part, T=_log(rng, 1, 1024), k=min(E, rng.randint(1, 8)), E=E, N=_log(rng, 64, 1024),
                K=16 * _log(rng, 4, 64), out=BF16 if part == "gate_up" else rng.choice([BF16, F32]))


# ---- inputs -----------------------------------------------------------------------------

def _routing(case, g):
    """Expert of each slot, int32 [T, k]: distinct per token, some experts likelier than others;
    padded tokens hold -1."""
    T, k, E = case["T"], case["k"], case["E"]
    like = torch.randn(E, generator=g, device="cuda") * 0.5
    gumbel = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)))
    ids = (gumbel + like).topk(k, dim=1).indices.to(torch.int32)
    if case.get("drop"):
        pad = torch.rand(T, generator=g, device="cuda") < 0.125
        ids = torch.where(pad[:, None], torch.full_like(ids, -1), ids)
    return ids.contiguous()


def _maps(ids, E):
    """Expert offsets [E+1] and the row of each slot [T, k] (-1: no expert), int32."""
    flat = ids.reshape(-1).long()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=order.device)
    row = torch.where(valid, row, torch.full_like(row, -1))
    count = torch.zeros(E + 1, dtype=torch.int64, device=order.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([count.new_zeros(1), count[:E].cumsum(0)])
    return offsets.to(torch.int32), row.to(torch.int32).view_as(ids), order, key


def _weights(rows, K, g):
    """int8 codes [rows, K] and fp32 scales [rows] of N(0, 0.02) weights."""
    w = torch.randn(rows, K, generator=g, device="cuda", dtype=torch.float32).mul_(0.02)
    s = w.abs().amax(1) / 127
    q = w.div_(s[:, None]).round_().clamp_(-127, 127).to(torch.int8)
    return q, s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1))

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    st = {"case": case}
    op = case["op"]
    if op in ("dispatch", "combine", "grad"):
        T, k, E, H, dt = case["T"], case["k"], case["E"], case["H"], DT[case["dtype"]]
        ids = _routing(case, g)
        if op == "dispatch":
            # a serving loop keeps its buffers; rows behind the last expert's keep what they held
            st.update(ids=ids, x=randn(T, H, dtype=dt), xs=torch.zeros(T * k, H, dtype=dt, device="cuda"))
        else:
            _, rows, _, _ = _maps(ids, E)
            w = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
            st.update(rows=rows, w=w, ys=randn(T * k, H, dtype=dt))
            if op == "grad":
                st.update(dy=randn(T, H, dtype=DT[case["out"]]), dxs=randn(T * k, H, dtype=dt),
                          dys=torch.zeros(T * k, H, dtype=dt, device="cuda"))
        return st
    N, K = case["N"], case["K"]
    if op == "i8":
        q, s = _weights(N, K, g)
        st.update(x=randn(case["M"], K), q=[q], s=[s])
    else:
        E, mats = case["E"], 2 if case["part"] == "gate_up" else 1
        ids = _routing(case, g)
        off, _, _, _ = _maps(ids, E)
        qs = [_weights(E * N, K, g) for _ in range(mats)]
        st.update(x=randn(case["T"] * case["k"], K), off=off, max_rows=int((off[1:] - off[:-1]).max()),
                  q=[q for q, _ in qs], s=[s for _, s in qs])
    if own:
        # the weights as a program loads them once: int8 checkpoints into the packed layout
        from block_quantized_weight_qgemm_b200 import qgemm

        if op == "i8":
            st["packed"] = qgemm.i8_repack_rowmajor(st["q"][0], st["s"][0])
        else:
            st["packed"] = [qgemm.I8ExpertTable([qgemm.i8_repack_rowmajor(q[e * N:(e + 1) * N], s[e * N:(e + 1) * N])
                                                 for e in range(case["E"])]) for q, s in zip(st["q"], st["s"])]
    return st


# ---- one pass ---------------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"dispatch": _dispatch, "combine": _combine, "grad": _grad, "i8": _i8, "i8_moe": _i8_moe}[st["case"]["op"]](st)


def _run_own(st):
    from block_quantized_weight_qgemm_b200 import qgemm

    case = st["case"]
    op = case["op"]
    if op == "dispatch":
        xs, offsets, rows = qgemm.moe_dispatch(st["x"], st["ids"], case["E"], xs=st["xs"])
        return {"xs": xs, "offsets": offsets, "rows": rows}
    if op == "combine":
        return {"y": qgemm.moe_combine(st["ys"], st["rows"], st["w"], y_dtype=DT[case["out"]])}
    if op == "grad":
        dys, dw = qgemm.moe_combine_grad(st["dy"], st["ys"], st["rows"], st["w"], dys=st["dys"])
        return {"dys": dys, "dw": dw, "dx": qgemm.moe_dispatch_grad(st["dxs"], st["rows"], dx_dtype=DT[case["out"]])}
    if op == "i8":
        return {"y": qgemm.i8_run(st["x"], st["packed"], y_dtype=DT[case["out"]])}
    if case["part"] == "gate_up":
        return {"h": qgemm.i8_moe_gate_up(st["x"], st["off"], st["packed"][0], st["packed"][1], st["max_rows"])}
    return {"y": qgemm.i8_moe_run(st["x"], st["off"], st["packed"][0], st["max_rows"], y_dtype=DT[case["out"]])}


def _dispatch(st):
    k, E = st["case"]["k"], st["case"]["E"]
    offsets, rows, order, key = _maps(st["ids"], E)
    x = st["x"][order // k]
    return {"xs": torch.where((key[order] < E)[:, None], x, torch.zeros_like(x)), "offsets": offsets, "rows": rows}


def _gathered(a, rows):
    """fp32 [T, k, H]: the rows of each token's slots, zeros for a slot without an expert."""
    r = a[rows.clamp(min=0).long()].float()
    return torch.where((rows >= 0)[:, :, None], r, torch.zeros_like(r))


def _combine(st):
    return {"y": (_gathered(st["ys"], st["rows"]) * st["w"][:, :, None]).sum(1).to(DT[st["case"]["out"]])}


def _grad(st):
    case, rows, w, dy = st["case"], st["rows"], st["w"], st["dy"].float()
    S, H = rows.numel(), case["H"]
    d = (dy[:, None, :] * w[:, :, None]).to(DT[case["dtype"]]).reshape(S, H)
    dys = d.new_zeros(S + 1, H)  # the last row takes what has no expert
    dys[torch.where(rows >= 0, rows, torch.full_like(rows, S)).reshape(-1).long()] = d
    dw = (dy[:, None, :] * _gathered(st["ys"], rows)).sum(2)
    return {"dys": dys[:S], "dw": dw, "dx": _gathered(st["dxs"], rows).sum(1).to(DT[case["out"]])}


def _quant(x):
    """Codes (fp32 values) and fp32 scales of bf16 rows; the rounding is decided in 64 bits."""
    s = x.float().abs().amax(1) / 127
    q = (x.double() / torch.where(s > 0, s, torch.ones_like(s)).double()[:, None]).round().clamp(-127, 127)
    return q.float(), s


def _i8(st):
    q, s = _quant(st["x"])
    acc = q @ st["q"][0].float().t()
    return {"y": (acc * st["s"][0][None, :] * s[:, None]).to(DT[st["case"]["out"]])}


def _i8_moe(st):
    case, off, R = st["case"], st["off"].long(), st["max_rows"]
    E, N, K = case["E"], case["N"], case["K"]
    q, s = _quant(st["x"])
    # the rows of each expert, padded to the longest: [E, R, K]
    at = off[:-1, None] + torch.arange(R, device=off.device)[None, :]
    has = at < off[1:, None]
    src = torch.where(has, at, torch.zeros_like(at))
    xe, se = q[src], s[src]
    outs = [torch.bmm(xe, w.view(E, N, K).float().transpose(1, 2)) * sw.view(E, 1, N) * se[:, :, None]
            for w, sw in zip(st["q"], st["s"])]
    o = outs[0] if case["part"] == "run" else outs[0] / (1 + torch.exp(-outs[0])) * outs[1]
    M = st["x"].shape[0]
    y = torch.empty(M + 1, N, dtype=DT[case["out"]], device=o.device)  # the last row takes the padding
    y[torch.where(has, at, torch.full_like(at, M)).reshape(-1)] = o.reshape(-1, N).to(y.dtype)
    return {("y" if case["part"] == "run" else "h"): y[:M]}


# ---- the definitions in 64 bits ---------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        # the rows as a list: token of every valid slot, by expert, then by slot
        ids = st["ids"].cpu().tolist()
        slots = sorted((e, t, j) for t, r in enumerate(ids) for j, e in enumerate(r) if e >= 0)
        xs = torch.zeros(st["xs"].shape, dtype=torch.float64, device="cuda")
        if slots:
            xs[:len(slots)] = st["x"].double()[torch.tensor([t for _, t, _ in slots], device="cuda")]
        return {"xs": xs, "offsets": None, "rows": None}
    if op in ("combine", "grad"):
        rows, w = st["rows"].long(), st["w"].double()
        T, k = rows.shape
        live = (rows >= 0).double()
        H = case["H"]
        if op == "combine":
            y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
            for j in range(k):
                y += st["ys"].double()[rows[:, j].clamp(min=0)] * (w[:, j] * live[:, j])[:, None]
            return {"y": y}
        dys = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        dx = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        dy = st["dy"].double()
        for j in range(k):
            t = torch.nonzero(rows[:, j] >= 0).reshape(-1)
            r = rows[t, j]
            dys[r] = dy[t] * w[t, j, None]
            dw[t, j] = (dy[t] * st["ys"].double()[r]).sum(1)
            dx[t] += st["dxs"].double()[r]
        return {"dys": dys, "dw": dw, "dx": dx}
    x = st["x"].double()
    s = (x.abs().amax(1).float() / 127.0).double()
    q = torch.where(s[:, None] > 0, torch.round(x / s[:, None]), torch.zeros_like(x)).clamp(-127, 127)
    if op == "i8":
        N = case["N"]
        y = torch.empty(case["M"], N, dtype=torch.float64, device="cuda")
        for n in range(0, N, 4096):
            y[:, n:n + 4096] = torch.matmul(q, st["q"][0][n:n + 4096].double().t()) * st["s"][0][n:n + 4096].double()
        return {"y": y * s[:, None]}
    N = case["N"]
    off = st["off"].cpu().tolist()
    y = torch.empty(x.shape[0], N, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        p = [torch.matmul(q[a:b], w[e * N:(e + 1) * N].double().t()) * sw[e * N:(e + 1) * N].double() * s[a:b, None]
             for w, sw in zip(st["q"], st["s"])]
        y[a:b] = p[0] if case["part"] == "run" else p[0] * torch.sigmoid(p[0]) * p[1]
    return {("y" if case["part"] == "run" else "h"): y}


def work(case):
    op, es = case["op"], 2 if case.get("dtype") == BF16 else 4
    eo = 2 if case.get("out") == BF16 else 4
    if op in ("dispatch", "combine", "grad"):
        T, H, E = case["T"], case["H"], case["E"]
        S = T * case["k"]
        live = 0.875 * S if case["drop"] else S  # padded tokens' rows are neither read nor written
        if op == "dispatch":
            return {"bytes": live / case["k"] * H * es + live * H * es + 8 * S + 4 * (E + 1), "flops": 0}
        if op == "combine":
            return {"bytes": live * H * es + T * H * eo + 8 * S, "flops": 2 * live * H}
        return {"bytes": 2 * T * H * eo + 3 * live * H * es + 16 * S, "flops": 4 * live * H}
    N, K = case["N"], case["K"]
    if op == "i8":
        M = case["M"]
        return {"bytes": 2 * M * K + N * K + 4 * N + M * N * eo, "flops": 2 * M * N * K}
    S, E, mats = case["T"] * case["k"], case["E"], 2 if case["part"] == "gate_up" else 1
    used = E * (1 - (1 - case["k"] / E) ** case["T"])  # experts that some token chose, about
    return {"bytes": 2 * S * K + used * mats * (N * K + 4 * N) + S * N * eo + 4 * (E + 1), "flops": 2 * mats * S * N * K}
