"""Timed cases of the batch-decoding operators, each with its plain form.

Three operators serve a batch of sequences that continue one prompt:

* "rope": RMSNorm of every query and key head, rotation by position, values
  rounded, in one pass over the projection's rows (``tf.qk_norm_rope``);
* "kv": rows written into a KV cache, as bf16 or quantised to 8 bits (E4M3 codes
  with one power-of-two scale per vector), and read back (``tf.KVBatch.store`` /
  ``load``);
* "attn": attention of each sequence's rows over the prompt's shared entries and
  the sequence's own (``tf.KVBatch.attention``).

``run`` makes one pass over what ``prepare`` gives: the framework's calls where
``own`` is true, elementary torch operations in fp32 where it is false.
"""

import math

import torch

own = False

D = 128           # head dimension
EPS = 1e-6
THETA = 1e6


def listed():
    return [
        # one row of one sequence: the serial decode step, all latency
        dict(name="rope_one_row", op="rope", seqs=1, rows=1, n_q=64, n_kv=8, rot=128, pairs="halves", fp32=True,
             start=70001),
        # a verify pass of 24 sequences x 5 rows
        dict(name="rope_verify", op="rope", seqs=24, rows=5, n_q=64, n_kv=8, rot=128, pairs="halves", fp32=True,
             start=8192),
        # an odd-sized prompt of bf16 rows, half of each head rotated in adjacent pairs
        dict(name="rope_prompt", op="rope", seqs=1, rows=16383, n_q=32, n_kv=4, rot=64, pairs="adjacent", fp32=False,
             start=0),
        # the new entries of a verify pass of 24 sequences
        dict(name="kv_verify", op="kv", seqs=24, rows=5, n_kv=8, fmt="e4m3", start=701),
        # a whole prompt written and read back
        dict(name="kv_prompt", op="kv", seqs=1, rows=32767, n_kv=8, fmt="e4m3", start=0),
        # three short replies to a short prompt: all latency
        dict(name="attn_short", op="attn", seqs=3, rows=1, n_kv=2, group=4, prefix=300, own_max=40, fmt="bf16", idle=0),
        # one serial sequence with no shared prompt
        dict(name="attn_alone", op="attn", seqs=1, rows=1, n_kv=8, group=8, prefix=0, own_max=2500, fmt="bf16", idle=0),
        # 32 replies decoding one token each, lengths ragged, two of them finished
        dict(name="attn_decode", op="attn", seqs=32, rows=1, n_kv=8, group=8, prefix=8192, own_max=700, fmt="bf16",
             idle=2),
        # 16 replies verifying five rows each over an 8-bit cache
        dict(name="attn_verify8", op="attn", seqs=16, rows=5, n_kv=8, group=8, prefix=16461, own_max=600, fmt="e4m3",
             idle=0),
        # few replies to a very long document, an odd head layout
        dict(name="attn_document", op="attn", seqs=4, rows=3, n_kv=4, group=5, prefix=130001, own_max=300, fmt="bf16",
             idle=0),
        # many replies verifying eight rows each: bound by the products
        dict(name="attn_wide", op="attn", seqs=64, rows=8, n_kv=8, group=8, prefix=32768, own_max=500, fmt="bf16",
             idle=1),
        # many replies over an 8-bit cache
        dict(name="attn_wide8", op="attn", seqs=60, rows=4, n_kv=8, group=8, prefix=20000, own_max=900, fmt="e4m3",
             idle=0),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "kv", "attn", "attn"])
    if op == "rope":
        seqs = _log(rng, 1, 96)
        n_kv = rng.choice([1, 2, 4, 8])
        return dict(op=op, seqs=seqs, rows=_log(rng, 1, max(16, 16384 // seqs)), n_q=n_kv * rng.choice([1, 2, 4, 5, 8]),
                    n_kv=n_kv, rot=rng.choice([32, 64, 96, 128]), pairs=rng.choice(["halves", "adjacent"]),
                    fp32=rng.random() < 0.5, start=rng.randrange(0, 1 << 20))
    if op == "kv":
        seqs = _log(rng, 1, 96)
        return dict(op=op, seqs=seqs, rows=_log(rng, 1, max(16, 32768 // seqs)), n_kv=rng.choice([1, 2, 4, 8]),
                    fmt=rng.choice(["e4m3", "e4m3", "bf16"]), start=rng.randrange(0, 1000))
    group = rng.choice([1, 2, 3, 4, 5, 8])
    n_kv = rng.choice([1, 2, 4, 8])
    seqs = _log(rng, 1, 64)
    rows = rng.choice([1, 1, 2, 3, 5, 8, 16]) if group <= 8 else 1
    prefix = _log(rng, 1, 131072) if rng.random() < 0.9 else 0
    own_max = _log(rng, 16, 2000)
    while seqs * rows * group * n_kv * (prefix + own_max) > 64 * 8 * 64 * 32768:
        prefix //= 2
    return dict(op=op, seqs=seqs, rows=rows, n_kv=n_kv, group=group, prefix=prefix, own_max=max(own_max, rows),
                fmt=rng.choice(["bf16", "e4m3"]), idle=1 if seqs > 2 and rng.random() < 0.3 else 0)


def _positions(case):
    """Position of each sequence's first row; -1 where the sequence is idle."""
    B, R = case["seqs"], case["rows"]
    if case["op"] == "rope":
        return [case["start"] + 37 * (b % 11) for b in range(B)]
    if case["op"] == "kv":
        return [case["start"] + (13 * b) % 29 for b in range(B)]
    longest = case["own_max"]   # entries of the longest sequence, its new rows included
    at = [longest - R if b == 0 else (7919 * b + 31) % (longest - R + 1) for b in range(B)]
    for i in range(case["idle"]):
        at[B - 1 - i] = -1
    return at


def _capacity(case):
    need = max(_positions(case)) + case["rows"]
    return -(-need // 256) * 256


def work(case):
    B, R = case["seqs"], case["rows"]
    if case["op"] == "rope":
        heads = case["n_q"] + 2 * case["n_kv"]
        n = B * R * heads * D
        return {"bytes": n * ((4 if case["fp32"] else 2) + 2), "flops": 10 * n}
    if case["op"] == "kv":
        n = 2 * B * R * case["n_kv"] * D
        held = 1 + 1 / D if case["fmt"] == "e4m3" else 2
        return {"bytes": n * (2 + 2 * held + 2), "flops": 4 * n}
    n_q = case["n_kv"] * case["group"]
    held = 1 + 1 / D if case["fmt"] == "e4m3" else 2
    active = [p for p in _positions(case) if p >= 0]
    entries = case["prefix"] + sum(p + R for p in active)
    seen = sum(case["prefix"] + p + r + 1 for p in active for r in range(R))
    return {"bytes": 2 * entries * case["n_kv"] * D * held + 4 * B * R * n_q * D, "flops": 4 * D * n_q * seen}


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B, R, n_kv = case["seqs"], case["rows"], case["n_kv"]
    pos = torch.tensor(_positions(case), dtype=torch.int64, device="cuda")
    s = dict(case=case, pos=pos)
    if case["op"] == "rope":
        heads = case["n_q"] + 2 * n_kv
        x = torch.randn((B * R, heads * D), generator=g, device="cuda") * 3
        s["x"] = x if case["fp32"] else x.to(torch.bfloat16)
        s["wq"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        s["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        if own:
            from w4_gemm_keyed_gb300 import tf
            s["turns"] = tf.rope_turns(case["rot"], THETA)
        else:
            s["inv_freq"] = THETA ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        return s
    if case["op"] == "kv":
        # vectors of very different sizes, some values far above the rest
        size = torch.exp2(torch.randint(-6, 7, (B * R, n_kv, 1), generator=g, device="cuda").float())
        s["k"] = (_normal(g, B * R, n_kv, D).float() * size).to(torch.bfloat16).reshape(B * R, n_kv * D)
        s["v"] = _normal(g, B * R, n_kv * D)
        if own:
            from w4_gemm_keyed_gb300 import tf
            s["cache"] = tf.KVBatch(B, n_kv, _capacity(case), case["fmt"])
            s["ws"] = tf.workspace(256)
        else:
            s["cache"] = _plain_cache(B, n_kv, _capacity(case), case["fmt"])
        return s
    n_q, L, P = n_kv * case["group"], _capacity(case), case["prefix"]
    s["q"] = (2 * torch.randn((B * R, n_q * D), generator=g, device="cuda")).to(torch.bfloat16)
    shared_k, shared_v = _normal(g, P, n_kv * D), _normal(g, P, n_kv * D)
    own_k, own_v = _normal(g, B * L, n_kv * D), _normal(g, B * L, n_kv * D)
    first, begin = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda")
    if own:
        from w4_gemm_keyed_gb300 import tf
        s["cache"] = tf.KVBatch(B, n_kv, L, case["fmt"])
        s["cache"].store(own_k, own_v, begin)
        s["prefix"] = None
        if P:
            s["prefix"] = tf.KVBatch(1, n_kv, -(-P // 256) * 256, case["fmt"])
            s["prefix"].store(shared_k, shared_v, first)
        s["ws"] = tf.workspace(s["cache"].attention_workspace_bytes(case["group"], R, P))
    else:
        s["cache"] = _plain_cache(B, n_kv, L, case["fmt"])
        _plain_store(s["cache"], own_k, own_v, begin)
        s["prefix"] = _plain_cache(1, n_kv, P, case["fmt"])
        if P:
            _plain_store(s["prefix"], shared_k, shared_v, first)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_cache(n_seq, n_kv, length, fmt):
    """Entries [n_seq][n_kv][length][128]: bf16 values, or E4M3 codes and their exponents."""
    def half():
        if fmt == "bf16":
            return dict(values=torch.zeros((n_seq, n_kv, length, D), dtype=torch.bfloat16, device="cuda"))
        return dict(codes=torch.zeros((n_seq, n_kv, length, D), dtype=torch.float8_e4m3fn, device="cuda"),
                    exponents=torch.zeros((n_seq, n_kv, length, 1), dtype=torch.int32, device="cuda"))
    return dict(k=half(), v=half(), n_seq=n_seq, n_kv=n_kv)


def _power(e):
    """2^e in fp32 for whole numbers e in [-126, 127], exact (pow need not be)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """E4M3 codes and power-of-two exponents of the vectors x [..., 128] (fp32): the
    smallest exponent e in [-120, 7] with max |x| <= 448 * 2^e."""
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))   # max = m * 2^e, m in [0.5, 1)
    e = torch.clamp(e - 9 + (m > 0.875).to(e.dtype), -120, 7)
    e = torch.where(m == 0, torch.full_like(e, -120), e)
    scaled = (x * _power(-e)).clamp(-448, 448)
    return scaled.to(torch.float8_e4m3fn), e


def _plain_store(cache, k, v, pos):
    n_seq, n_kv = cache["n_seq"], cache["n_kv"]
    R = k.shape[0] // n_seq
    seq = torch.arange(n_seq, device="cuda").repeat_interleave(R)
    at = (pos[:, None] + torch.arange(R, device="cuda")).reshape(-1)
    for half, rows in ((cache["k"], k), (cache["v"], v)):
        rows = rows.reshape(n_seq * R, n_kv, D)
        if "values" in half:
            half["values"][seq, :, at] = rows
        else:
            codes, e = _quantise(rows.float())
            half["codes"].view(torch.uint8)[seq, :, at] = codes.view(torch.uint8)
            half["exponents"][seq, :, at] = e


def _plain_values(half):
    """fp32 values of a half of a plain cache."""
    if "values" in half:
        return half["values"].float()
    return half["codes"].float() * _power(half["exponents"])


def _plain_load(cache, pos, R):
    n_seq, n_kv = cache["n_seq"], cache["n_kv"]
    seq = torch.arange(n_seq, device="cuda").repeat_interleave(R)
    at = (pos[:, None] + torch.arange(R, device="cuda")).reshape(-1)
    got = []
    for half in (cache["k"], cache["v"]):
        if "values" in half:
            rows = half["values"][seq, :, at]
        else:
            codes = half["codes"].view(torch.uint8)[seq, :, at].view(torch.float8_e4m3fn)
            rows = (codes.float() * _power(half["exponents"][seq, :, at])).to(torch.bfloat16)
        got.append(rows.reshape(n_seq * R, n_kv * D))
    return got


def _plain_rope(s):
    case = s["case"]
    rows, n_q, n_kv, rot = s["x"].shape[0], case["n_q"], case["n_kv"], case["rot"]
    x = s["x"].float().reshape(rows, n_q + 2 * n_kv, D)
    qk, v = x[:, :n_q + n_kv], x[:, n_q + n_kv:]
    w = torch.cat([s["wq"].float().expand(n_q, D), s["wk"].float().expand(n_kv, D)])
    qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + EPS) * w
    at = (s["pos"][:, None] + torch.arange(case["rows"], device="cuda")).reshape(-1)
    angle = torch.remainder(at.double()[:, None] * s["inv_freq"], 2 * math.pi)     # far positions need 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if case["pairs"] == "halves":
        a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    y = torch.cat([torch.cat([turned, qk[..., rot:]], -1), v], 1)
    return y.to(torch.bfloat16).reshape(rows, -1)


def _plain_attention(s):
    case = s["case"]
    B, R, n_kv, g = case["seqs"], case["rows"], case["n_kv"], case["group"]
    q = s["q"].float().reshape(B, R, n_kv, g, D) / math.sqrt(D)
    own_k, own_v = _plain_values(s["cache"]["k"]), _plain_values(s["cache"]["v"])
    shared_k, shared_v = _plain_values(s["prefix"]["k"])[0], _plain_values(s["prefix"]["v"])[0]
    by_head = q.permute(2, 0, 1, 3, 4).reshape(n_kv, B * R * g, D)
    by_seq = q.permute(0, 2, 1, 3, 4).reshape(B, n_kv, R * g, D)
    a = by_head @ shared_k.transpose(1, 2)                                       # [n_kv][B R g][prefix]
    b = by_seq @ own_k.transpose(2, 3)                                           # [B][n_kv][R g][own]
    last = s["pos"][:, None] + torch.arange(R, device="cuda")                    # last entry each row sees
    last = torch.where(s["pos"][:, None] < 0, torch.full_like(last, -1), last)
    hidden = torch.arange(own_k.shape[2], device="cuda") > last[..., None]       # [B][R][own]
    hidden = hidden.repeat_interleave(g, 1)[:, None]
    b = b.masked_fill(hidden, float("-inf"))
    b = b.reshape(B, n_kv, R, g, -1).permute(1, 0, 2, 3, 4).reshape(n_kv, B * R * g, -1)
    top = b.amax(-1, keepdim=True)
    if case["prefix"]:
        top = torch.maximum(top, a.amax(-1, keepdim=True))
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    a, b = torch.exp(a - top), torch.exp(b - top)
    total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    o = a @ shared_v
    b = b.reshape(n_kv, B, R * g, -1).transpose(0, 1)
    o = o + (b @ own_v).transpose(0, 1).reshape(n_kv, B * R * g, D)
    o = o / total
    idle = (s["pos"] < 0).repeat_interleave(R * g)[None, :, None]
    o = torch.where(idle, torch.zeros_like(o), o)
    return o.reshape(n_kv, B * R, g, D).transpose(0, 1).reshape(B * R, n_kv * g * D).to(torch.bfloat16)


def run(s):
    case = s["case"]
    if own:
        from w4_gemm_keyed_gb300 import tf
        if case["op"] == "rope":
            return tf.qk_norm_rope(s["x"], case["n_q"], case["n_kv"], s["pos"], turns=s["turns"], q_weight=s["wq"],
                                   k_weight=s["wk"], eps=EPS, adjacent=case["pairs"] == "adjacent")
        if case["op"] == "kv":
            s["cache"].store(s["k"], s["v"], s["pos"], ws=s["ws"])
            return s["cache"].load(s["pos"], case["rows"], ws=s["ws"])
        return s["cache"].attention(s["q"], case["group"], s["pos"], prefix=s["prefix"], prefix_len=case["prefix"],
                                    ws=s["ws"])
    if case["op"] == "rope":
        return _plain_rope(s)
    if case["op"] == "kv":
        _plain_store(s["cache"], s["k"], s["v"], s["pos"])
        return _plain_load(s["cache"], s["pos"], case["rows"])
    return _plain_attention(s)


# ---------------------------------------------------------------- 64 bits
def _e4m3_nearest(x):
    """x (fp64 vectors) as the nearest E4M3 value times its vector's power of two, ties to even."""
    def two(e):
        return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)

    peak = x.abs().amax(-1, keepdim=True)
    unit = two(torch.full_like(peak, -120))
    for e in range(-119, 8):   # the smallest power of two with peak <= 448 of it
        unit = torch.where(peak > 448 * unit, two(torch.full_like(peak, e)), unit)
    y = x / unit
    # spacing of E4M3 at y: 2^(floor(log2 |y|) - 3), at least 2^-9
    step = two(torch.clamp(torch.frexp(y)[1] - 4, min=-9))
    return torch.clamp(torch.round(y / step) * step, -448, 448) * unit


def exact(case, seed):
    """What ``run`` returns, from the definitions in fp64."""
    global own
    kept, own = own, False
    s = prepare(case, seed)
    own = kept
    B, R, n_kv = case["seqs"], case["rows"], case["n_kv"]
    if case["op"] == "kv":
        rows = [s["k"].double().reshape(-1, D), s["v"].double().reshape(-1, D)]
        if case["fmt"] == "e4m3":
            rows = [_e4m3_nearest(x) for x in rows]
        return [x.reshape(B * R, n_kv * D) for x in rows]
    if case["op"] == "rope":
        n_q, rot = case["n_q"], case["rot"]
        x = s["x"].double().reshape(B * R, n_q + 2 * n_kv, D).clone()
        for h0, h1, w in ((0, n_q, s["wq"]), (n_q, n_q + n_kv, s["wk"])):
            h = x[:, h0:h1]
            x[:, h0:h1] = h / (h.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
        row = torch.arange(B * R, device="cuda")
        p = (s["pos"][row // R] + row % R).double()
        y = x.clone()
        for i in range(rot // 2):
            i0, i1 = (i, i + rot // 2) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)
            angle = (p * THETA ** (-2 * i / rot))[:, None]
            a, b = x[:, :n_q + n_kv, i0], x[:, :n_q + n_kv, i1]
            y[:, :n_q + n_kv, i0] = a * angle.cos() - b * angle.sin()
            y[:, :n_q + n_kv, i1] = b * angle.cos() + a * angle.sin()
        return y.reshape(B * R, -1)
    g, P = case["group"], case["prefix"]
    if work(case)["flops"] > 1.5e12:
        return None
    held = [[_plain_values(c[h]).double() for h in ("k", "v")] for c in (s["prefix"], s["cache"])]
    q = s["q"].double().reshape(B, R, n_kv, g, D)
    out = torch.zeros_like(q)
    for b, p in enumerate(_positions(case)):
        if p < 0:
            continue
        for j in range(n_kv):
            k = torch.cat([held[0][0][0, j], held[1][0][b, j, :p + R]])
            v = torch.cat([held[0][1][0, j], held[1][1][b, j, :p + R]])
            z = torch.einsum("rhd,td->rht", q[b, :, j], k) * D ** -0.5
            t = torch.arange(k.shape[0], device="cuda")
            late = t[None, :] > P + p + torch.arange(R, device="cuda")[:, None]
            weight = torch.softmax(z.masked_fill(late[:, None], -math.inf), -1)
            out[b, :, j] = torch.einsum("rht,td->rhd", weight, v)
    return out.reshape(B * R, n_kv * g * D)
