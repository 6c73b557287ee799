"""Measured cases of the operators around a Muon step's inputs.

A Muon step reads one gradient per hidden matrix, and QK-Clip reads the largest
attention logit of each head. These operators produce both:

  checkpoint     an activation is held in 8 bits until the backward pass (int8 values, one
                 power-of-two scale per token and 32 columns) and restored there
  weight_grad    dW = dY^T X of a hidden matrix, or of a stack of experts, with X read from
                 its 8-bit checkpoint
  attention      softmax attention of packed sequences, with the log-sum-exp of each row and
                 the largest logit of each head
  attention_bwd  its backward pass, which recomputes the probabilities from the log-sum-exp

`run` computes them in elementary torch operations, or with `own` set by the library.
"""
import math

import torch

own = False

F32, BF16 = "float32", "bfloat16"
GROUP = 32           # columns that share one scale of a checkpoint
DTYPES = {F32: torch.float32, BF16: torch.bfloat16}


def _nums(text):
    return [int(x) for x in text.split(",")]


def _text(values):
    return ",".join(str(int(v)) for v in values)


# ---------------------------------------------------------------- cases
def listed():
    """The listed cases. Widths come from the library's shape sets (hidden 512, 768, 1024 and
    2048; experts of 320; an MLP of 5632); sequence lengths are those of packed training
    batches."""
    # a batch of documents packed to 8192 tokens: many short ones, a few long ones
    docs = "2311,37,1024,640,1,1503,255,129,512,980,800"
    # 8192 tokens x 4 experts each over 64 experts: a skewed router, two experts without tokens
    counts = [1487, 0, 911, 300, 512, 77, 640, 1024] + [512 + 37 * ((i * 29) % 17 - 8) for i in range(55)]
    counts += [0]
    return [
        # the latency of a call: one token of a 2048-wide model
        dict(name="checkpoint_one_token", op="checkpoint", rows=1, cols=2048, ld=2048, dtype=BF16),
        # an odd width in 32 bits: columns that end inside a group and a vector
        dict(name="checkpoint_odd_f32", op="checkpoint", rows=777, cols=1021, ld=1021, dtype=F32),
        # the MLP activation of a 1.5B model, 16384 tokens
        dict(name="checkpoint_mlp", op="checkpoint", rows=16384, cols=5632, ld=5632, dtype=BF16),
        # a short last micro-batch: few tokens into a square projection, gradient in 32 bits
        dict(name="wgrad_few_tokens", op="weight_grad", out=768, inn=768, counts="97", dtype=F32),
        # long accumulation into a small matrix: the token axis is all the parallelism there is
        dict(name="wgrad_long_small", op="weight_grad", out=512, inn=320, counts="16384", dtype=F32),
        # the MLP matrix of a 1.5B model, 8192 tokens
        dict(name="wgrad_mlp", op="weight_grad", out=5632, inn=2048, counts="8192", dtype=BF16),
        # the up projections of 64 experts of 320 in a 512-wide model
        dict(name="wgrad_experts", op="weight_grad", out=320, inn=512, counts=_text(counts), dtype=BF16),
        # three short sequences: a call's latency, rows of one key
        dict(name="attention_short", op="attention", lengths="1,17,130", k_lengths="1,17,130", heads=8,
             kv_heads=8, dim=128, causal=True),
        # a packed batch of documents in a 2048-wide model, four query heads to a key head
        dict(name="attention_packed", op="attention", lengths=docs, k_lengths=docs, heads=16,
             kv_heads=4, dim=128, causal=True),
        # one long sequence in a 768-wide model, every key visible
        dict(name="attention_long_full", op="attention", lengths="8191", k_lengths="8191", heads=12,
             kv_heads=12, dim=64, causal=False),
        # the backward passes of a packed batch and of one long causal sequence
        dict(name="attention_bwd_packed", op="attention_bwd", lengths=docs, k_lengths=docs, heads=12,
             kv_heads=12, dim=64, causal=True),
        dict(name="attention_bwd_long", op="attention_bwd", lengths="8192", k_lengths="8192", heads=16,
             kv_heads=4, dim=128, causal=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _split(rng, total, parts, floor=0):
    """`parts` ragged lengths of at least `floor` that add up to `total`."""
    w = [rng.expovariate(1.0) for _ in range(parts)]
    left = total - floor * parts
    out = [floor + int(left * x / sum(w)) for x in w]
    out[rng.randrange(parts)] += total - sum(out)
    return out


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["checkpoint", "weight_grad", "attention", "attention_bwd"])
    top = max((c for c in listed() if c["op"] == op), key=_cost)
    while True:
        if op == "checkpoint":
            cols = _log_int(rng, 1, 6144)
            c = dict(op=op, rows=_log_int(rng, 1, 16384), cols=cols, ld=cols + rng.choice([0, 0, 8, 5]),
                     dtype=rng.choice([F32, BF16]))
        elif op == "weight_grad":
            experts = rng.choice([1, 1, _log_int(rng, 2, 64)])
            tokens = _log_int(rng, 1, 32768)
            counts = [tokens] if experts == 1 else _split(rng, tokens, experts)
            c = dict(op=op, out=_log_int(rng, 8, 6144), inn=_log_int(rng, 8, 6144), counts=_text(counts),
                     dtype=rng.choice([F32, BF16]))
        else:
            kv = rng.choice([1, 2, 4, 8])
            n = rng.choice([1, 1, _log_int(rng, 2, 16)])
            total = _log_int(rng, n, 8192)
            lens = _split(rng, total, n, 1)
            # keys: as many as queries, or another number (a prefix that needs no gradient of its own)
            k_lens = lens if rng.random() < 0.7 else [max(0, x + rng.randint(-x, 256)) for x in lens]
            if sum(k_lens) == 0:
                continue
            c = dict(op=op, lengths=_text(lens), k_lengths=_text(k_lens), heads=kv * rng.choice([1, 2, 4]),
                     kv_heads=kv, dim=rng.choice([64, 128, 128, 96]), causal=rng.random() < 0.7)
        if _cost(c) <= _cost(top) and _size(c) <= _size(top):
            return c


def _cost(case):
    w = work(case)
    return w["flops"] / 50e12 + w["bytes"] / 3e12


def _size(case):
    return work(case)["bytes"] if case["op"] in ("checkpoint", "weight_grad") else 0


def _pairs(case):
    """Visible query-key pairs of one head. Causal rows are aligned at the end of the keys:
    query i of m sees key j of n when j <= i + n - m."""
    total = 0
    for m, n in zip(_nums(case["lengths"]), _nums(case["k_lengths"])):
        if not case["causal"]:
            total += m * n
        else:
            rows = min(m, n)                       # rows that see at least one key
            total += rows * n - rows * (rows - 1) // 2
    return total


def work(case):
    op = case["op"]
    if op == "checkpoint":
        elem = case["rows"] * case["cols"]
        size = 4 if case["dtype"] == F32 else 2
        groups = case["rows"] * ((case["cols"] + GROUP - 1) // GROUP)
        return {"bytes": 2 * (elem * size + elem + groups), "flops": 6 * elem}
    if op == "weight_grad":
        counts = _nums(case["counts"])
        t, o, i = sum(counts), case["out"], case["inn"]
        size = 4 if case["dtype"] == F32 else 2
        return {"bytes": t * o * 2 + t * i + t * ((i + GROUP - 1) // GROUP) + len(counts) * o * i * size,
                "flops": 2 * t * o * i}
    m, n = sum(_nums(case["lengths"])), sum(_nums(case["k_lengths"]))
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    q_rows, k_rows = m * h * d * 2, n * g * d * 2
    if op == "attention":
        return {"bytes": 2 * q_rows + 2 * k_rows + 4 * m * h + 4 * h, "flops": 4 * d * h * _pairs(case)}
    return {"bytes": 4 * q_rows + 4 * k_rows + 4 * m * h, "flops": 10 * d * h * _pairs(case)}


# ---------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _padded(rows, cols, ld, dtype):
    """A rows x cols view of a buffer with leading dimension ld."""
    return torch.zeros(rows, ld, device="cuda", dtype=dtype)[:, :cols]


def _activation(gen, rows, cols, ld, dtype):
    """Activations with a few strong channels, as hidden states have them."""
    gain = torch.exp(0.8 * _normal(gen, 1, cols))
    x = _padded(rows, cols, ld, dtype)
    x.copy_(_normal(gen, rows, cols) * gain)
    return x


def _quantise(x):
    """The checkpoint's values and scales, in elementary operations: the scale of a group of
    32 columns is 2^(e - 6), 2^e <= largest magnitude < 2^(e + 1), and at least 2^-126."""
    rows, cols = x.shape
    pad = -cols % GROUP
    x = torch.nn.functional.pad(x.float(), (0, pad)).view(rows, -1, GROUP)
    top = x.abs().amax(2, keepdim=True)
    e = torch.frexp(top)[1] - 7                                 # frexp: top = f 2^k, 1/2 <= f < 1
    e = torch.where(top > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    q = torch.round(torch.ldexp(x.double(), -e)).clamp(-127, 127)
    return q, e


def _restore(q, e, cols):
    return torch.ldexp(q.double(), e).float().flatten(1)[:, :cols]


def _offsets(lengths):
    off = [0]
    for n in lengths:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def _up(n, k):
    return (n + k - 1) // k * k


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if own:
        from matrix_orthogonalising_optimizer_03_b200 import binding as B
        st["B"] = B
    if op == "checkpoint":
        st["x"] = _activation(gen, case["rows"], case["cols"], case["ld"], DTYPES[case["dtype"]])
        if own:
            st["ck"] = B.new_act8(case["rows"], case["cols"])
            st["y"] = torch.empty_like(st["x"])
        return st
    if op == "weight_grad":
        counts, o, i = _nums(case["counts"]), case["out"], case["inn"]
        t = sum(counts)
        x = _activation(gen, t, i, i, torch.bfloat16)
        dy = _padded(t, o, _up(o, 8), torch.bfloat16)
        dy.copy_(_normal(gen, t, o) * 1e-3 * torch.exp(0.5 * _normal(gen, t, 1)))
        st["dy"] = dy
        st["offsets"] = _offsets(counts)
        q, e = _quantise(x)
        if own:
            ck = B.new_act8(t, i)
            ck.q[:, :i].copy_(q.flatten(1)[:, :i])               # the same stored values for both sides
            ck.exps[:, :e.shape[1]].copy_(e.squeeze(2) + 127)
            st["dw"] = torch.empty(len(counts), o, i, device="cuda", dtype=DTYPES[case["dtype"]])
            st["plan"] = B.WeightGradPlan(dy, ck, st["dw"], offsets=st["offsets"])
        else:
            st["q"] = q.to(torch.int8).flatten(1)[:, :i].contiguous()
            st["scale"] = torch.ldexp(torch.ones((), device="cuda"), e.squeeze(2))
        return st
    m, n = sum(_nums(case["lengths"])), sum(_nums(case["k_lengths"]))
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    # heads of different sharpness: logits of a few units, more in some heads
    gain = torch.exp(0.4 * _normal(gen, 1, g, 1))
    st["q"] = (_normal(gen, m, h, d) * 1.2).bfloat16()
    st["k"] = (_normal(gen, n, g, d) * gain).bfloat16()
    st["v"] = _normal(gen, n, g, d).bfloat16()
    st["q_off"], st["k_off"] = _offsets(_nums(case["lengths"])), _offsets(_nums(case["k_lengths"]))
    if op == "attention_bwd":
        st["dout"] = (_normal(gen, m, h, d) * 1e-2).bfloat16()
        st["o"], st["lse"], _ = _plain_attention(st)            # what the forward pass left
    if own:
        kw = dict(q_offsets=st["q_off"], k_offsets=st["k_off"], causal=case["causal"])
        if op == "attention":
            st["o"] = torch.empty_like(st["q"])
            st["lse"] = torch.empty(h, m, device="cuda")
            st["s_max"] = torch.empty(h, device="cuda")
            st["plan"] = B.AttentionPlan(st["q"], st["k"], st["v"], st["o"], st["lse"], s_max=st["s_max"], **kw)
        else:
            for x in ("q", "k", "v"):
                st["d" + x] = torch.empty_like(st[x])
            st["plan"] = B.AttentionPlan(st["q"], st["k"], st["v"], st["o"], st["lse"],
                                         grads=(st["dout"], st["dq"], st["dk"], st["dv"]), **kw)
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        if op == "checkpoint":
            state["B"].act8_store([state["x"]], [state["ck"]])
            state["B"].act8_restore([state["ck"]], [state["y"]])
            return state["y"]
        if op == "weight_grad":
            state["plan"].apply()
            return state["dw"]
        if op == "attention":
            state["s_max"].fill_(-math.inf)                      # forward() raises it: a step starts it anew
            state["plan"].forward()
            return state["o"], state["lse"], state["s_max"]
        state["plan"].backward()
        return state["dq"], state["dk"], state["dv"]
    if op == "checkpoint":
        q, e = _quantise(state["x"])
        return _restore(q.to(torch.int8), e, state["case"]["cols"]).to(state["x"].dtype)
    if op == "weight_grad":
        return _plain_weight_grad(state)
    if op == "attention":
        return _plain_attention(state)
    return _plain_attention_bwd(state)


def _plain_weight_grad(state):
    case = state["case"]
    counts, i = _nums(case["counts"]), case["inn"]
    x = state["q"].float() * state["scale"].repeat_interleave(GROUP, 1)[:, :i]
    dy = state["dy"].float()
    dw = torch.zeros(len(counts), case["out"], i, device="cuda")
    lo = 0
    for g, n in enumerate(counts):
        if n:
            dw[g] = dy[lo:lo + n].t() @ x[lo:lo + n]
        lo += n
    return dw.to(DTYPES[case["dtype"]])


def _visible(m, n, causal, r0, r1):
    """Mask of the keys that rows r0..r1 of m queries see among n keys."""
    i = torch.arange(r0, r1, device="cuda").unsqueeze(1)
    j = torch.arange(n, device="cuda")
    return (j <= i + (n - m)) if causal else torch.ones(r1 - r0, n, dtype=torch.bool, device="cuda")


def _spans(case):
    """Per sequence its rows and keys, and per key head its query heads."""
    q0 = k0 = 0
    for m, n in zip(_nums(case["lengths"]), _nums(case["k_lengths"])):
        yield q0, q0 + m, k0, k0 + n
        q0, k0 = q0 + m, k0 + n


def _plain_attention(state):
    case = state["case"]
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    q, k, v = state["q"], state["k"], state["v"]
    o = torch.zeros(q.shape, device="cuda")
    lse = torch.full((h, q.shape[0]), -math.inf, device="cuda")
    s_max = torch.full((h,), -math.inf, device="cuda")
    for q0, q1, k0, k1 in _spans(case):
        if q1 == q0 or k1 == k0:
            continue
        mask = _visible(q1 - q0, k1 - k0, case["causal"], 0, q1 - q0)
        for kh in range(g):
            hs = slice(kh * (h // g), (kh + 1) * (h // g))
            s = q[q0:q1, hs].float().transpose(0, 1) @ k[k0:k1, kh].float().t() / math.sqrt(d)
            s = torch.where(mask, s, -math.inf)
            top = s.amax(2, keepdim=True)
            s_max[hs] = torch.maximum(s_max[hs], top.amax((1, 2)))
            p = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
            tot = p.sum(2, keepdim=True)
            lse[hs, q0:q1] = (top + torch.log(tot)).squeeze(2)
            o[q0:q1, hs] = ((p @ v[k0:k1, kh].float()) / torch.where(tot > 0, tot, 1.0)).transpose(0, 1)
    return o.bfloat16(), lse, s_max


def _plain_attention_bwd(state):
    case = state["case"]
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    q, k, v, o, do, lse = (state[x] for x in ("q", "k", "v", "o", "dout", "lse"))
    dq, dk, dv = (torch.zeros(x.shape, device="cuda") for x in (q, k, v))
    delta = (o.float() * do.float()).sum(2).t()                  # heads x rows
    for q0, q1, k0, k1 in _spans(case):
        if q1 == q0 or k1 == k0:
            continue
        mask = _visible(q1 - q0, k1 - k0, case["causal"], 0, q1 - q0)
        for kh in range(g):
            hs = slice(kh * (h // g), (kh + 1) * (h // g))
            qf, dof = q[q0:q1, hs].float().transpose(0, 1), do[q0:q1, hs].float().transpose(0, 1)
            kf, vf = k[k0:k1, kh].float(), v[k0:k1, kh].float()
            s = qf @ kf.t() / math.sqrt(d)
            p = torch.where(mask, torch.exp(s - lse[hs, q0:q1].unsqueeze(2)), 0.0)
            dv[k0:k1, kh] = (p.transpose(1, 2) @ dof).sum(0)
            ds = p * (dof @ vf.t() - delta[hs, q0:q1].unsqueeze(2)) / math.sqrt(d)
            dq[q0:q1, hs] = (ds @ kf).transpose(0, 1)
            dk[k0:k1, kh] = (ds.transpose(1, 2) @ qf).sum(0)
    return dq.bfloat16(), dk.bfloat16(), dv.bfloat16()


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op == "checkpoint":
        x = st["x"].double()
        y = torch.empty_like(x)
        for c0 in range(0, x.shape[1], GROUP):
            part = x[:, c0:c0 + GROUP]
            top = part.abs().amax(1, keepdim=True)
            low = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -120))))
            step = torch.where(2 * low <= top, 2 * low, low) / 64    # log2 of a power of two may fall short
            y[:, c0:c0 + GROUP] = torch.minimum(torch.maximum(torch.round(part / step), -127 * torch.ones_like(step)),
                                                127 * torch.ones_like(step)) * step
        return y
    if op == "weight_grad":
        out, lo = [], 0
        scale = st["scale"].double()
        for n in _nums(case["counts"]):
            x = st["q"][lo:lo + n].double()
            for c0 in range(0, case["inn"], GROUP):
                x[:, c0:c0 + GROUP] *= scale[lo:lo + n, c0 // GROUP:c0 // GROUP + 1]
            out.append(torch.einsum("to,ti->oi", st["dy"][lo:lo + n].double(), x))
            lo += n
        return torch.stack(out)
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    q, k, v = (st[x].double() for x in ("q", "k", "v"))
    o, s_max = torch.zeros_like(q), torch.full((h,), -math.inf, device="cuda", dtype=torch.float64)
    lse = torch.full((h, q.shape[0]), -math.inf, device="cuda", dtype=torch.float64)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for q0, q1, k0, k1 in _spans(case):
        if q1 == q0 or k1 == k0:
            continue
        for a in range(h):
            kh = a // (h // g)
            for r0 in range(q0, q1, 4096):
                r1 = min(q1, r0 + 4096)
                mask = _visible(q1 - q0, k1 - k0, case["causal"], r0 - q0, r1 - q0)
                s = torch.einsum("id,jd->ij", q[r0:r1, a], k[k0:k1, kh]) * d ** -0.5
                s = s.masked_fill(~mask, -math.inf)
                if op == "attention":
                    lse[a, r0:r1] = torch.logsumexp(s, 1)
                    s_max[a] = torch.maximum(s_max[a], s.max())
                    p = torch.exp(s - lse[a, r0:r1, None]).masked_fill(~mask, 0.0)
                    o[r0:r1, a] = torch.einsum("ij,jd->id", p, v[k0:k1, kh])
                    continue
                do = st["dout"][r0:r1, a].double()
                p = torch.exp(s - st["lse"][a, r0:r1, None].double()).masked_fill(~mask, 0.0)
                dv[k0:k1, kh] += torch.einsum("ij,id->jd", p, do)
                t = torch.einsum("id,jd->ij", do, v[k0:k1, kh])
                t = p * (t - torch.einsum("id,id->i", st["o"][r0:r1, a].double(), do)[:, None]) * d ** -0.5
                dq[r0:r1, a] = torch.einsum("ij,jd->id", t, k[k0:k1, kh])
                dk[k0:k1, kh] += torch.einsum("ij,id->jd", t, q[r0:r1, a])
    return (o, lse, s_max) if op == "attention" else (dq, dk, dv)
