"""The fp8 and router-training operators: their cases, plain forms and work.

Five operators of the library are described here, one case naming one of them
in ``"op"``:

* ``balance``   the router's balance loss with its per-expert counts, and the
                gradient of the logits (one pass is forward and backward)
* ``quantize``  rows or 128 x 128 blocks to e4m3 codes with a scale per 128
* ``matmul``    the product of two e4m3 operands with block scales
* ``gate_up``   the experts' gate|up product over routed rows, GLU, and the
                result quantised again
* ``down``      the experts' down product over sorted rows

``run`` computes them in elementary torch operations, in fp32, or, where the
module's ``own`` is set, by the library's calls. ``exact`` is the definition in
fp64, written apart from both.
"""
import math
from types import SimpleNamespace

import torch

own = False

DEV = "cuda"
BLOCK = 128
MAXQ = 448.0              # the largest e4m3 value
TINY = 2.0 ** -100        # groups below this magnitude take its scale

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a micro-batch of the small top-2 layer: latency counts
        dict(name="balance 64x8", op="balance", T=64, E=8, k=2, seqs=1, masked=False),
        # a training batch of ragged sequences with padding inside and behind them
        dict(name="balance 65521x256 ragged", op="balance", T=65521, E=256, k=8, seqs=13,
             masked=True),
        # the one token of a decode step, before the experts
        dict(name="quantize 1x2048 bf16", op="quantize", rows=1, K=2048, block=1, dtype="bf16"),
        # the token rows of a large prefill chunk
        dict(name="quantize 4096x7168 f16", op="quantize", rows=4096, K=7168, block=1,
             dtype="f16"),
        # eight experts' gate|up weights turned into the fp8 format at load time
        dict(name="quantize 8x11264x2048 f32 blocks", op="quantize", rows=8 * 11264, K=2048,
             block=128, dtype="f32"),
        # a dense (shared-expert) product of one decoded token
        dict(name="matmul 1x4096x7168", op="matmul", M=1, N=4096, K=7168, dtype="bf16"),
        # a small batch, sizes that end inside every tile
        dict(name="matmul 77x1000x2064", op="matmul", M=77, N=1000, K=2064, dtype="f32"),
        # the shared expert of a prefill chunk
        dict(name="matmul 4096x4096x7168", op="matmul", M=4096, N=4096, K=7168, dtype="bf16"),
        # one decoded token through 8 of 128 experts
        dict(name="gate_up 1 of 128x768", op="gate_up", T=1, E=128, k=8, d=2048, F=768,
             act="swiglu"),
        # a 2,048-token prefill chunk over 512 experts (20,480 routed rows)
        dict(name="gate_up 2048 of 512x512", op="gate_up", T=2048, E=512, k=10, d=2048, F=512,
             act="swiglu"),
        # 32 decoded tokens over 128 experts: one to five rows each
        dict(name="down 32 of 128x768", op="down", T=32, E=128, k=8, d=2048, F=768,
             act="swiglu"),
        # large experts, many rows each: bound by the tensor cores
        dict(name="down 4096 of 8x5632", op="down", T=4096, E=8, k=2, d=2048, F=5632,
             act="swiglu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "quantize", "matmul", "gate_up", "down"])
    if op == "balance":
        E = _log_int(rng, 4, 1024)
        T = _log_int(rng, 1, min(65536, 16_000_000 // E))
        k = rng.randint(1, min(E, 16))
        return dict(op=op, T=T, E=E, k=k, seqs=_log_int(rng, 1, 24), masked=rng.random() < 0.5)
    if op == "quantize":
        K = 16 * _log_int(rng, 8, 1024)
        rows = _log_int(rng, 1, 60_000_000 // K)
        return dict(op=op, rows=rows, K=K, block=rng.choice([1, 1, 128]),
                    dtype=rng.choice(sorted(_DTYPES)))
    if op == "matmul":
        N = _log_int(rng, 64, 8192)
        K = 16 * _log_int(rng, 8, 512)
        M = _log_int(rng, 1, min(8192, 100_000_000_000 // (N * K)))
        return dict(op=op, M=M, N=N, K=K, dtype=rng.choice(sorted(_DTYPES)))
    E = rng.choice([8, 16, 32, 64, 100, 128, 256])
    d = 128 * rng.randint(2, 24)
    F = 128 * rng.randint(1, max(1, min(16, 500_000_000 // (E * d * 256))))
    k = rng.randint(1, 8)
    T = _log_int(rng, 1, max(1, min(4096, 40_000_000_000 // (k * d * F))))
    return dict(op=op, T=T, E=E, k=k, d=d, F=F, act=rng.choice(["swiglu", "swiglu", "geglu"]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _weights(g, E, rows, K):
    """e4m3 codes [E, rows, K] and scales [E, ceil(rows/128), ceil(K/128)] of
    weights N(0, 1/K): a 128 x 128 block of them has its largest magnitude near
    four standard deviations, so that its codes are spread like 100 N(0, 1)."""
    q = torch.empty(E, rows, K, dtype=F8, device=DEV)
    step = max(1, 200_000_000 // (rows * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.randn(n, rows, K, generator=g, device=DEV, dtype=torch.float32)
        q[e:e + n] = w.mul_(100).clamp_(-MAXQ, MAXQ).to(F8)
    s = torch.rand(E, -(-rows // BLOCK), -(-K // BLOCK), generator=g, device=DEV)
    return q, (0.8 + 0.4 * s) / (100 * math.sqrt(K))


def _activations(g, rows, K):
    """e4m3 codes [rows, K] and scales [rows, ceil(K/128)] of rows whose
    magnitudes differ by an order."""
    x = torch.randn(rows, K, generator=g, device=DEV)
    x *= torch.exp(torch.randn(rows, 1, generator=g, device=DEV))
    return _quantize(x, 1)


def _tables(g, T, E, k):
    """The dispatch tables of k distinct experts per token, experts of uneven
    popularity, as the sort by expert gives them; and the most rows of one."""
    keys = torch.randn(T, E, generator=g, device=DEV)
    keys += 0.5 * torch.randn(1, E, generator=g, device=DEV)
    idx = keys.topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(idx, stable=True).indices
    inv = torch.empty_like(order)
    inv[order] = torch.arange(T * k, device=DEV)
    counts = torch.zeros(E, dtype=torch.int64, device=DEV).scatter_add_(
        0, idx, torch.ones_like(idx))
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    roff = torch.cat([zero, counts.cumsum(0)])
    toff = torch.cat([zero, ((counts + BLOCK - 1) // BLOCK).cumsum(0)])
    u32 = lambda t: t.to(torch.int32).view(torch.uint32)  # noqa: E731
    return dict(order=u32(order), inv_order=u32(inv), row_map=u32(order // k),
                counts=counts.int(), row_off=roff.int(), tile_off=toff.int()), int(counts.max())


def prepare(case, seed):
    g = _gen(seed)
    c, op = case, case["op"]
    st = dict(case=dict(case))
    if op == "balance":
        T, E, k, B = c["T"], c["E"], c["k"], c["seqs"]
        logits = torch.randn(T, E, generator=g, device=DEV)
        logits += 0.5 * torch.randn(1, E, generator=g, device=DEV)
        st["idx"] = logits.topk(k, dim=1).indices.int()
        st["mask"] = st["seq_off"] = None
        if c["masked"]:
            st["mask"] = torch.rand(T, generator=g, device=DEV) < 0.9
            # padding: nobody has written anything sensible there
            logits[~st["mask"]] = float("nan")
        if B > 1:
            # B sequences of random lengths, tokens behind the last one
            cuts = torch.rand(B, generator=g, device=DEV).mul(T + 1).long().sort().values
            st["seq_off"] = torch.cat([torch.zeros_like(cuts[:1]), cuts]).clamp_(max=T).int()
        st["logits"] = logits
        st["coef"] = 0.01
        st["dloss"] = torch.ones((), device=DEV)
        return st
    if op == "quantize":
        x = torch.randn(c["rows"], c["K"], generator=g, device=DEV)
        x *= torch.exp(torch.randn(c["rows"], 1, generator=g, device=DEV))
        st["x"] = x.to(_DTYPES[c["dtype"]])
        return st
    if op == "matmul":
        st["a"], st["sa"] = _activations(g, c["M"], c["K"])
        b, sb = _weights(g, 1, c["N"], c["K"])
        st["b"], st["sb"] = b[0], sb[0]
        return st
    T, E, k, d, F = c["T"], c["E"], c["k"], c["d"], c["F"]
    st["tables"], st["most"] = _tables(g, T, E, k)
    ex = SimpleNamespace(fmt="f8", E=E, d=d, F=F, act=c["act"], w_gu=None, s_gu=None, b_gu=None,
                         w_dn=None, s_dn=None, b_dn=None)
    if op == "gate_up":
        st["x"], st["xs"] = _activations(g, T, d)
    else:
        st["h"], st["hs"] = _activations(g, T * k, F)
    ex.w_gu, ex.s_gu = _weights(g, E, 2 * F, d)
    ex.w_dn, ex.s_dn = _weights(g, E, d, F)
    st["experts"] = ex
    return st


# ------------------------------------------------------------------ plain forms

def _blocks(x):
    """x [..., K] in groups of 128 along K, the last one filled with zeros."""
    K = x.shape[-1]
    pad = -K % BLOCK
    if pad:
        x = torch.nn.functional.pad(x, (0, pad))
    return x.unflatten(-1, (-1, BLOCK))


def _codes(x, amax):
    return torch.where(torch.isfinite(x), x * (MAXQ / amax), float("nan")).to(F8)


def _magnitude(x):
    return torch.where(torch.isfinite(x), x.abs(), 0.0)


def _quantize(x, block):
    x = x.float()
    rows, K = x.shape
    xb = _blocks(x)                                      # [rows, K/128, 128]
    amax = _magnitude(xb).amax(-1)
    if block == 1:
        amax = amax.clamp_min(TINY)
        return _codes(xb, amax[..., None]).flatten(1)[:, :K].contiguous(), amax / MAXQ
    amax = torch.nn.functional.pad(amax, (0, 0, 0, -rows % BLOCK))
    amax = amax.unflatten(0, (-1, BLOCK)).amax(1).clamp_min(TINY)
    each = amax.repeat_interleave(BLOCK, 0)[:rows]
    return _codes(xb, each[..., None]).flatten(1)[:, :K].contiguous(), amax / MAXQ


def _values(q, s):
    """fp32 values of codes [..., K] with scales [..., ceil(K/128)]."""
    K = q.shape[-1]
    return (_blocks(q.float()) * s[..., None]).flatten(-2)[..., :K]


def _weight_values(q, s):
    """fp32 values of codes [..., N, K] with a scale per 128 x 128 block."""
    N = q.shape[-2]
    return _values(q, s.repeat_interleave(BLOCK, -2)[..., :N, :])


def _plain_balance(st):
    lg, idx, mask, off = st["logits"], st["idx"].long(), st["mask"], st["seq_off"]
    T, E = lg.shape
    k = idx.shape[1]
    B = 1 if off is None else off.numel() - 1
    t = torch.arange(T, device=lg.device)
    seq = torch.zeros_like(t) if off is None else \
        torch.searchsorted(off.long(), t, right=True) - 1
    valid = (seq >= 0) & (seq < B)
    if mask is not None:
        valid &= mask
    seq = seq.clamp(0, B - 1)
    p = torch.where(valid[:, None], torch.softmax(lg, 1), 0.0)
    one = (seq == torch.arange(B, device=lg.device)[:, None]) & valid       # [B, T]
    tokens = one.sum(1)
    counts = torch.zeros(B * E, dtype=torch.int64, device=lg.device).scatter_add_(
        0, (seq[:, None] * E + idx).reshape(-1),
        valid[:, None].expand(T, k).reshape(-1).long()).reshape(B, E)
    n = tokens.clamp_min(1).float()[:, None]
    probs = one.float() @ p / n
    loss = st["coef"] * E / (B * k) * (counts * probs / n).sum()
    a = (st["dloss"] * st["coef"] * E / (B * k)) * counts / (n * n)          # dL/dp [B, E]
    at = a[seq]
    d = p * (at - (at * p).sum(1, keepdim=True))
    return dict(loss=loss, counts=counts.int(), probs=probs, tokens=tokens.int(), dlogits=d)


def _group_index(st):
    """Where the sorted rows stand in a padded [experts with rows, most, ...]
    batch: the experts taken, the row of each place, the place of each row."""
    c = st["case"]
    roff = st["tables"]["row_off"].long()
    n, R = min(c["E"], c["T"] * c["k"]), c["T"] * c["k"]
    act = torch.sort(roff[1:] - roff[:-1], descending=True, stable=True).indices[:n]
    rank = torch.zeros(c["E"], dtype=torch.int64, device=DEV)
    rank[act] = torch.arange(n, device=DEV)
    rows = (roff[act][:, None] + torch.arange(st["most"], device=DEV)).clamp(max=R - 1)
    i = torch.arange(R, device=DEV)
    e = torch.searchsorted(roff, i, right=True) - 1
    return act, rows, rank[e] * st["most"] + i - roff[e]


def _glu(act, g, u):
    if act == "geglu":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) * u
    return g / (1 + torch.exp(-g)) * u


def _plain_gate_up(st):
    ex = st["experts"]
    act, rows, place = _group_index(st)
    x = _values(st["x"], st["xs"])
    tok = st["tables"]["row_map"].view(torch.int32).long()
    w = _weight_values(ex.w_gu[act], ex.s_gu[act])
    gu = torch.bmm(x[tok[rows]], w.transpose(1, 2)).flatten(0, 1)[place]
    return _quantize(_glu(ex.act, gu[:, :ex.F], gu[:, ex.F:]), 1)


def _plain_down(st):
    ex = st["experts"]
    act, rows, place = _group_index(st)
    h = _values(st["h"], st["hs"])
    w = _weight_values(ex.w_dn[act], ex.s_dn[act])
    return torch.bmm(h[rows], w.transpose(1, 2)).flatten(0, 1)[place].half()


# ------------------------------------------------------------------ run

def _tables_of(moe, st):
    return moe.SortTables(**st["tables"], BM=BLOCK)


def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if own:
        import sparse_mixture_experts_top_b200 as moe
    if op == "balance":
        if own:
            b = moe.balance_loss(st["logits"], st["idx"], st["coef"], mask=st["mask"],
                                 seq_off=st["seq_off"])
            d = moe.balance_loss_backward(st["logits"], b, c["k"], st["coef"], mask=st["mask"],
                                          seq_off=st["seq_off"], dloss=st["dloss"])
            return dict(loss=b.loss, counts=b.counts, probs=b.probs, tokens=b.tokens, dlogits=d)
        return _plain_balance(st)
    if op == "quantize":
        q, s = moe.quantize_fp8(st["x"], c["block"]) if own else _quantize(st["x"], c["block"])
        return dict(q=q, s=s)
    if op == "matmul":
        dt = _DTYPES[c["dtype"]]
        if own:
            return moe.fp8_matmul(st["a"], st["sa"], st["b"], st["sb"], dt)
        return (_values(st["a"], st["sa"]) @ _weight_values(st["b"], st["sb"]).t()).to(dt)
    if op == "gate_up":
        if own:
            q, s = moe.grouped_swiglu_fp8(st["x"], st["xs"], _tables_of(moe, st), c["k"],
                                          st["experts"])
        else:
            q, s = _plain_gate_up(st)
        return dict(q=q, s=s)
    if own:
        return moe.grouped_down_fp8(st["h"], st["hs"], _tables_of(moe, st), c["T"], c["k"],
                                    st["experts"])
    return _plain_down(st)


# ------------------------------------------------------------------ work

def work(case):
    c, op = case, case["op"]
    if op == "balance":
        # the logits and the selection read once, the gradient written once
        T, E = c["T"], c["E"]
        return dict(bytes=T * E * 8 + T * c["k"] * 4 + c["seqs"] * E * 8, flops=10 * T * E)
    if op == "quantize":
        n = c["rows"] * c["K"]
        groups = -(-c["rows"] // c["block"]) * -(-c["K"] // BLOCK)
        return dict(bytes=n * (_SIZE[c["dtype"]] + 1) + 4 * groups, flops=2 * n)
    if op == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        kb = -(-K // BLOCK)
        return dict(bytes=(M + N) * K + 4 * kb * (M + -(-N // BLOCK)) + M * N * _SIZE[c["dtype"]],
                    flops=2 * M * N * K)
    T, E, k, d, F = c["T"], c["E"], c["k"], c["d"], c["F"]
    R = T * k
    active = E * (1 - (1 - k / E) ** T)       # experts that some token takes, in the mean
    if op == "gate_up":
        return dict(bytes=active * 2 * F * d * (1 + 4 / BLOCK ** 2) + T * d * (1 + 4 / BLOCK) +
                    R * F * (1 + 4 / BLOCK) + 4 * R, flops=4 * R * d * F)
    return dict(bytes=active * F * d * (1 + 4 / BLOCK ** 2) + R * F * (1 + 4 / BLOCK) + R * d * 2,
                flops=2 * R * d * F)


# ------------------------------------------------------------------ exact

def _e4m3_of(v):
    """fp64 values rounded to the nearest e4m3 value, ties to even: three
    fraction bits, exponents from -6, the largest value 448."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -40))).clamp_min(-6)
    step = torch.pow(2.0, e - 3)
    return (torch.round(v / step) * step).clamp(-MAXQ, MAXQ)


def _exact_rows(x):
    """Codes and scales of finite fp64 rows, one scale per row and 128 columns."""
    q, s = [], []
    for k in range(0, x.shape[1], BLOCK):
        part = x[:, k:k + BLOCK]
        top = part.abs().max(1, keepdim=True).values.clamp_min(TINY)
        q.append(_e4m3_of(part * MAXQ / top))
        s.append(top / MAXQ)
    return torch.cat(q, 1), torch.cat(s, 1)


def _decoded(q, s, rows_per_scale):
    """fp64 values of a matrix of codes, block by block."""
    v = q.double()
    for k in range(0, v.shape[1], BLOCK):
        for i in ([slice(None)] if rows_per_scale == 1 else
                  [slice(j, j + BLOCK) for j in range(0, v.shape[0], BLOCK)]):
            f = s[i, k // BLOCK] if rows_per_scale == 1 else s[i.start // BLOCK, k // BLOCK]
            v[i, k:k + BLOCK] *= f.double()[:, None] if rows_per_scale == 1 else f.double()
    return v


def _exact_balance(st):
    lg = st["logits"].double()
    T, E = lg.shape
    k = st["idx"].shape[1]
    ok = torch.ones(T, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"]
    off = [0, T] if st["seq_off"] is None else st["seq_off"].tolist()
    B = len(off) - 1
    loss = torch.zeros((), dtype=torch.float64, device=DEV)
    probs = torch.zeros(B, E, dtype=torch.float64, device=DEV)
    d = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    for b in range(B):
        t = off[b] + ok[off[b]:off[b + 1]].nonzero().flatten()
        n = t.numel()
        if not n:
            continue
        z = torch.exp(lg[t] - lg[t].max(1, keepdim=True).values)
        p = z / z.sum(1, keepdim=True)
        f = torch.bincount(st["idx"][t].flatten().long(), minlength=E).double() * E / (k * n)
        probs[b] = p.sum(0) / n
        loss += st["coef"] / B * (f * probs[b]).sum()
        d[t] = float(st["dloss"]) * st["coef"] / (B * n) * p * (f - (p @ f)[:, None])
    return dict(loss=loss, counts=None, probs=probs, tokens=None, dlogits=d)


def _exact_experts(st):
    ex, tb = st["experts"], st["tables"]
    off = tb["row_off"].tolist()
    up = st["case"]["op"] == "gate_up"
    if up:
        src = _decoded(st["x"], st["xs"], 1)[tb["row_map"].view(torch.int32).long()]
    else:
        src = _decoded(st["h"], st["hs"], 1)
    out = torch.empty(off[-1], ex.F if up else ex.d, dtype=torch.float64, device=DEV)
    for e in range(ex.E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        v = src[a:b] @ _decoded((ex.w_gu if up else ex.w_dn)[e], (ex.s_gu if up else ex.s_dn)[e],
                                BLOCK).t()
        if up:
            g, u = v[:, :ex.F], v[:, ex.F:]
            if ex.act == "geglu":
                v = torch.nn.functional.gelu(g, approximate="tanh") * u
            else:
                v = torch.nn.functional.silu(g) * u
        out[a:b] = v
    if not up:
        return out
    q, s = _exact_rows(out)
    return dict(q=q, s=s)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "balance":
        return _exact_balance(st)
    if op == "quantize":
        x = st["x"].double()
        if case["block"] == 1:
            q, s = _exact_rows(x)
            return dict(q=q, s=s)
        q, rows = torch.empty_like(x), []
        for i in range(0, x.shape[0], BLOCK):
            part = x[i:i + BLOCK]
            row = []
            for k in range(0, x.shape[1], BLOCK):
                top = part[:, k:k + BLOCK].abs().max().clamp_min(TINY)
                q[i:i + BLOCK, k:k + BLOCK] = _e4m3_of(part[:, k:k + BLOCK] * MAXQ / top)
                row.append(top / MAXQ)
            rows.append(torch.stack(row))
        return dict(q=q, s=torch.stack(rows))
    if op == "matmul":
        return _decoded(st["a"], st["sa"], 1) @ _decoded(st["b"], st["sb"], BLOCK).t()
    return _exact_experts(st)
