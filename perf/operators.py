"""The measured cases of the gated linear recurrence, attention over prompts and attention over
a 4-bit cache: their inputs, their plain forms in elementary torch operations, the calls of
gated_delta_rule_kla_amd.kla that compute the same, and what they give in 64 bits.

Operators (a case's "op"):
  glr_fwd    h_t = exp(g_t) h_{t-1} + x_t per channel, over packed or dense sequences
  glr_bwd    its gradients for x, g and the initial state
  glr_step   one token per sequence, the state updated in place
  attn       causal softmax attention, grouped heads, packed sequences; with lq < lk a prompt
             that is continued after earlier keys (the last query sees the last key)
  kv4_store  keys and values put into the pages of a 4-bit cache, and the stored values read
             back (what a continued prompt attends to)
  kv4_decode one query per sequence over the paged 4-bit cache

The cache holds blocks of 32 channels as E2M1 codes (two to a byte, the even channel in the low
half) with a power-of-two scale per block (E8M0).
"""

import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
PAGE = 64


def listed():
    return [
        # a prefill of 4 x 4096 tokens through 16 heads of 128 channels
        {"name": "glr_fwd_prefill", "op": "glr_fwd", "dt": "bf16", "B": 4, "H": 16, "T": 4096, "d": 128, "lo": 0, "pack": 0, "seqs": 0},
        # one long document, 65,536 tokens: 4,096 channels and no other parallelism
        {"name": "glr_fwd_long", "op": "glr_fwd", "dt": "bf16", "B": 1, "H": 16, "T": 65536, "d": 256, "lo": 0, "pack": 0, "seqs": 0},
        # a training step's gradients over 32 packed documents of 512 to 16,384 tokens
        {"name": "glr_bwd_packed", "op": "glr_bwd", "dt": "bf16", "B": 1, "H": 16, "T": 0, "d": 128, "lo": 512, "pack": 16384, "seqs": 32},
        # the debug build's tiny fp32 shape: latency
        {"name": "glr_bwd_tiny", "op": "glr_bwd", "dt": "fp32", "B": 1, "H": 1, "T": 256, "d": 16, "lo": 0, "pack": 0, "seqs": 0},
        # one interactive user: a single token
        {"name": "glr_step_one", "op": "glr_step", "dt": "bf16", "N": 1, "H": 16, "d": 128},
        # a serving batch of 256 sequences
        {"name": "glr_step_batch", "op": "glr_step", "dt": "bf16", "N": 256, "H": 16, "d": 128},
        # a batch of prompts of different lengths, 16 query heads over 4 key heads
        {"name": "attn_packed", "op": "attn", "dt": "bf16", "B": 1, "seqs": 12, "lo": 200, "pack": 4096, "lq": 0, "lk": 0, "Hq": 16, "Hkv": 4, "D": 128},
        # one long prompt
        {"name": "attn_long", "op": "attn", "dt": "bf16", "B": 1, "seqs": 0, "lo": 0, "pack": 0, "lq": 16384, "lk": 16384, "Hq": 16, "Hkv": 2, "D": 128},
        # the keys of one new token for each of 256 sequences
        {"name": "kv4_store_step", "op": "kv4_store", "dt": "bf16", "seqs": 256, "lo": 1, "pack": 1, "before": 4000, "Hkv": 4, "D": 128},
        # the keys of 32 whole prompts
        {"name": "kv4_store_prompts", "op": "kv4_store", "dt": "bf16", "seqs": 32, "lo": 512, "pack": 16384, "before": 0, "Hkv": 4, "D": 128},
        # a serving batch of 64 sequences with up to 16,384 cached tokens
        {"name": "kv4_decode_batch", "op": "kv4_decode", "dt": "bf16", "seqs": 64, "lo": 4096, "pack": 16384, "Hq": 16, "Hkv": 4, "D": 128},
        # one user with a context of 131,072 tokens
        {"name": "kv4_decode_long", "op": "kv4_decode", "dt": "bf16", "seqs": 1, "lo": 131071, "pack": 131071, "Hq": 16, "Hkv": 2, "D": 128},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glr_fwd", "glr_bwd", "glr_step", "attn", "kv4_store", "kv4_decode"])
    dt = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("glr_fwd", "glr_bwd"):
        H, d = rng.choice([1, 2, 5, 16]), rng.choice([16, 64, 100, 128, 256, 1000, 2560])
        most = max(64, min(65536, (1 << 26) // (H * d)))  # tokens in all
        if rng.random() < 0.5:
            seqs = rng.randint(2, 24)
            top = max(8, most // seqs)
            return {"op": op, "dt": dt, "B": 1, "H": H, "T": 0, "d": d, "lo": max(1, top // 32), "pack": _log_int(rng, max(2, top // 16), top), "seqs": seqs}
        B = rng.choice([1, 1, 3, 8])
        return {"op": op, "dt": dt, "B": B, "H": H, "T": _log_int(rng, 1, max(8, most // B)), "d": d, "lo": 0, "pack": 0, "seqs": 0}
    if op == "glr_step":
        return {"op": op, "dt": dt, "N": _log_int(rng, 1, 512), "H": rng.choice([1, 3, 16, 32]), "d": rng.choice([16, 60, 128, 256, 1000])}
    Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    group = rng.choice([1, 2, 4, 5, 8])
    if op == "attn":
        if rng.random() < 0.5:
            return {"op": op, "dt": dt, "B": 1, "seqs": rng.randint(2, 12), "lo": rng.randint(1, 60), "pack": _log_int(rng, 100, 3000), "lq": 0, "lk": 0,
                    "Hq": Hkv * group, "Hkv": Hkv, "D": D}
        lq = _log_int(rng, 1, 3000)
        return {"op": op, "dt": dt, "B": rng.choice([1, 2]), "seqs": 0, "lo": 0, "pack": 0, "lq": lq, "lk": lq + rng.choice([0, 0, _log_int(rng, 1, 3000)]),
                "Hq": Hkv * group, "Hkv": Hkv, "D": D}
    if op == "kv4_store":
        seqs = _log_int(rng, 1, 64)
        top = _log_int(rng, 1, 4000)
        return {"op": op, "dt": dt, "seqs": seqs, "lo": max(1, top // 8), "pack": top, "before": rng.choice([0, rng.randint(1, 3000)]), "Hkv": Hkv, "D": D}
    seqs = _log_int(rng, 1, 128)
    top = _log_int(rng, 1, min(65536, 400000 // seqs))
    return {"op": op, "dt": dt, "seqs": seqs, "lo": max(1, top // 8), "pack": top, "Hq": Hkv * group, "Hkv": Hkv, "D": D}


def _lengths(case):
    """The case's own ragged lengths, log-uniform in [lo, pack]; they do not depend on the seed."""
    rng = random.Random(case["seqs"] * 1000003 + case["lo"] * 1009 + case["pack"])
    return [_log_int(rng, case["lo"], case["pack"]) if case["pack"] > case["lo"] else case["lo"] for _ in range(case["seqs"])]


def _bounds(lens, dev):
    host = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
    return host.to(dev), host


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, op = DT[case["dt"]], case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(std)

    def log_decay(*shape):  # slow decays, as a recurrence over long sequences has
        return torch.nn.functional.softplus(normal(*shape)).mul_(-0.1).to(dt)

    s = {"case": case}
    if op in ("glr_fwd", "glr_bwd"):
        B, H, T, d = (case[k] for k in ("B", "H", "T", "d"))
        N, s["cu"], s["cu_host"] = B, None, None
        if case["seqs"]:
            lens = _lengths(case)
            N, T = len(lens), sum(lens)
            s["cu"], s["cu_host"] = _bounds(lens, dev)
        s["x"], s["g"] = normal(B, H, T, d).to(dt), log_decay(B, H, T, d)
        s["h0"] = normal(N, H, d)
        if op == "glr_bwd":
            s["o"] = _glr_fwd(s)[0]  # the forward pass's output
            s["do"], s["dfinal"] = normal(B, H, T, d).to(dt), normal(N, H, d)
            del s["x"]
    elif op == "glr_step":
        N, H, d = (case[k] for k in ("N", "H", "d"))
        s["x"], s["g"], s["state"] = normal(N, H, d).to(dt), log_decay(N, H, d), normal(N, H, d)
    elif op == "attn":
        B, Hq, Hkv, D = (case[k] for k in ("B", "Hq", "Hkv", "D"))
        lq, lk, s["cu"], s["cu_host"] = case["lq"], case["lk"], None, None
        if case["seqs"]:
            lens = _lengths(case)
            lq = lk = sum(lens)
            s["cu"], s["cu_host"] = _bounds(lens, dev)
        s["q"], s["k"], s["v"] = normal(B, Hq, lq, D).to(dt), normal(B, Hkv, lk, D).to(dt), normal(B, Hkv, lk, D).to(dt)
    else:
        Hkv, D = case["Hkv"], case["D"]
        lens = _lengths(case)
        before = case.get("before", 0)
        M = -(-(max(lens) + before) // PAGE)
        P = len(lens) * M + 3
        order = torch.randperm(P, generator=gen, device=dev)[: len(lens) * M]
        s["table"] = order.to(torch.int32).reshape(len(lens), M).contiguous()
        s["codes"] = torch.zeros(P, 2, Hkv, PAGE, D // 2, dtype=torch.uint8, device=dev)
        s["scales"] = torch.zeros(P, 2, Hkv, PAGE, D // 32, dtype=torch.uint8, device=dev)
        loud = 1 + 3 * (torch.rand(Hkv, 1, D, generator=gen, device=dev) < 0.03)  # a few channels of keys are large
        if op == "kv4_store":
            T = sum(lens)
            s["cu"], s["cu_host"] = _bounds(lens, dev)
            s["k"], s["v"] = (normal(1, Hkv, T, D) * loud).to(dt), normal(1, Hkv, T, D).to(dt)
            s["start"] = torch.full((len(lens),), before, dtype=torch.int32, device=dev)
        else:
            for p in range(0, P, 512):
                n = min(512, P - p)
                for j, m in ((0, loud), (1, 1.0)):
                    c, e = _quantise((normal(n, Hkv, PAGE, D) * m).to(torch.bfloat16).float())
                    s["codes"][p:p + n, j], s["scales"][p:p + n, j] = c, e
            s["q"] = normal(len(lens), case["Hq"], D).to(dt)
            s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
            s["max_len"] = max(lens)
    return s


# ---- the plain forms -------------------------------------------------------------------------


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 2, h_{-1} = 0, by doubling."""
    step, T = 1, a.shape[2]
    a, b = a.clone(), b.clone()
    while step < T:
        b[:, :, step:] = b[:, :, step:] + a[:, :, step:] * b[:, :, :-step]
        a[:, :, step:] = a[:, :, step:] * a[:, :, :-step]
        step *= 2
    return b


def _edges(s, T, B):
    """Row and token of each sequence's first and last token."""
    dev = s["g"].device
    if s["cu"] is None:
        row = torch.arange(B, device=dev)
        return row, torch.zeros_like(row), torch.full_like(row, T - 1)
    cu = s["cu"].long()
    return torch.zeros_like(cu[1:]), cu[:-1], cu[1:] - 1


def _glr_fwd(s):
    x, g, h0 = s["x"], s["g"], s["h0"]
    row, first, last = _edges(s, x.shape[2], x.shape[0])
    a, b = torch.exp(g.float()), x.float().clone()
    b[row, :, first] += a[row, :, first] * h0
    a[row, :, first] = 0.0
    h = _scan(a, b)
    return h.to(x.dtype), h[row, :, last].contiguous()


def _glr_bwd(s):
    g, o, do, h0 = s["g"], s["o"], s["do"], s["h0"]
    row, first, last = _edges(s, g.shape[2], g.shape[0])
    a, b = torch.exp(g.float()), do.float().clone()
    b[row, :, last] += s["dfinal"]
    after = torch.zeros_like(a)  # the decay of the next token, none behind a sequence's last
    after[:, :, :-1] = a[:, :, 1:]
    after[row, :, last] = 0.0
    dh = _scan(after.flip(2), b.flip(2)).flip(2)
    prev = torch.zeros_like(a)
    prev[:, :, 1:] = o[:, :, :-1].float()
    prev[row, :, first] = h0
    dh0 = a[row, :, first] * dh[row, :, first]
    return dh.to(g.dtype), (dh * a * prev).to(g.dtype), dh0


def _glr_step(s):
    s["state"].copy_(torch.exp(s["g"].float()) * s["state"] + s["x"].float())
    return s["state"].to(s["x"].dtype), s["state"]


def _attn(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, Hq, Tq, D = q.shape
    group = Hq // k.shape[1]
    cu = [0, Tq] if s["cu"] is None else s["cu_host"].tolist()
    off = k.shape[2] - Tq
    out = torch.empty(B, Hq, Tq, D, dtype=q.dtype, device=q.device)
    lse = torch.empty(B, Hq, Tq, dtype=torch.float32, device=q.device)
    for b in range(B):
        for a, z in zip(cu, cu[1:]):
            ends = torch.arange(a, z, device=q.device)[:, None] + off
            mask = torch.arange(a, z + off, device=q.device)[None, :] > ends
            for h in range(Hq):
                sc = q[b, h, a:z].float() @ k[b, h // group, a:z + off].float().T
                sc = sc.mul_(D ** -0.5).masked_fill_(mask, float("-inf"))
                top = sc.max(1, keepdim=True).values
                p = sc.sub_(top).exp_()
                tot = p.sum(1, keepdim=True)
                out[b, h, a:z] = ((p @ v[b, h // group, a:z + off].float()) / tot).to(q.dtype)
                lse[b, h, a:z] = (top + torch.log(tot))[:, 0]
    return out, lse


def _quantise(x):
    """E2M1 codes (packed) and E8M0 scales of x [..., D] in fp32, blocks of 32 along D."""
    blocks = x.unflatten(-1, (-1, 32))
    top = blocks.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -126).clamp(-126, 127)
    y = blocks * torch.exp2(-e.float())[..., None]
    m = y.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code + 8 * (y < 0)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _values(codes, scales, dtype=torch.float32):
    """The values that codes [..., D/2] and scales [..., D/32] stand for."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=dtype, device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    e = torch.exp2(scales.to(dtype) - 127)
    return (v.unflatten(-1, (-1, 32)) * e[..., None]).flatten(-2)


def _places(s):
    """Page and place in it of every token of the packed keys."""
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n, output_size=s["k"].shape[2])
    pos = torch.arange(s["k"].shape[2], device=n.device) - s["cu"].long()[seq] + s["start"].long()[seq]
    return s["table"][seq, pos // PAGE].long(), pos % PAGE


def _kv4_store(s):
    page, at = _places(s)
    both = []
    for j, x in enumerate((s["k"], s["v"])):
        codes, scales = _quantise(x[0].float())
        s["codes"][page, j, :, at] = codes.transpose(0, 1)
        s["scales"][page, j, :, at] = scales.transpose(0, 1)
    for j in (0, 1):
        x = _values(s["codes"][page, j, :, at], s["scales"][page, j, :, at])
        both.append(x.transpose(0, 1).to(s["k"].dtype).contiguous()[None])
    return both


def _kv4_decode(s, dtype=torch.float32):
    q, table = s["q"], s["table"].long()
    N, Hq, D = q.shape
    Hkv = s["codes"].shape[2]
    there = torch.arange(table.shape[1] * PAGE, device=q.device)[None] < s["lens"][:, None]
    kv = [_values(s["codes"][table, j], s["scales"][table, j]).transpose(1, 2).reshape(N, Hkv, -1, D) for j in (0, 1)]
    sc = q.float().view(N, Hkv, Hq // Hkv, D) @ kv[0].transpose(2, 3).contiguous() * D ** -0.5
    sc = sc.masked_fill(~there[:, None, None], float("-inf"))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    return ((p @ kv[1]) / p.sum(-1, keepdim=True)).reshape(N, Hq, D).to(q.dtype)


PLAIN = {"glr_fwd": _glr_fwd, "glr_bwd": _glr_bwd, "glr_step": _glr_step, "attn": _attn, "kv4_store": _kv4_store,
         "kv4_decode": _kv4_decode}


# ---- the framework's calls ---------------------------------------------------------------------


def _calls(s):
    from gated_delta_rule_kla_amd import kla

    op = s["case"]["op"]
    if op == "glr_fwd":
        return kla.glr_chunk_fwd(s["x"], s["g"], s["h0"], s["cu"], cu_seqlens_host=s["cu_host"])
    if op == "glr_bwd":
        return kla.glr_chunk_bwd(s["g"], s["o"], s["do"], s["h0"], s["dfinal"], s["cu"], cu_seqlens_host=s["cu_host"])
    if op == "glr_step":
        return kla.glr_decode_step(s["x"], s["g"], s["state"]), s["state"]
    if op == "attn":
        return kla.attn_fwd(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], cu_seqlens_host=s["cu_host"])
    if op == "kv4_store":
        kla.kv4_append(s["k"], s["v"], s["codes"], s["scales"], s["table"], s["start"], s["cu"], cu_seqlens_host=s["cu_host"])
        return kla.kv4_read(s["codes"], s["scales"], s["table"], s["start"], s["cu"], s["k"].dtype, cu_seqlens_host=s["cu_host"])
    return kla.attn_kv4_decode_step(s["q"], s["codes"], s["scales"], s["table"], s["lens"], max_len=s["max_len"])


def run(s):
    return _calls(s) if own else PLAIN[s["case"]["op"]](s)


# ---- what a pass cannot do without -----------------------------------------------------------------


def work(case):
    op, e = case["op"], 2 if case["dt"] == "bf16" else 4
    lens = _lengths(case) if case.get("seqs") else []
    if op in ("glr_fwd", "glr_bwd"):
        n = case["H"] * case["d"] * (sum(lens) if lens else case["B"] * case["T"])
        states = (len(lens) or case["B"]) * case["H"] * case["d"] * 4
        return {"bytes": (3 if op == "glr_fwd" else 5) * n * e + (2 if op == "glr_fwd" else 3) * states, "flops": (2 if op == "glr_fwd" else 5) * n}
    if op == "glr_step":
        n = case["N"] * case["H"] * case["d"]
        return {"bytes": 3 * n * e + 8 * n, "flops": 2 * n}
    if op == "attn":
        if lens:
            tq = tk = sum(lens)
            pairs = sum(n * (n + 1) // 2 for n in lens)
        else:
            tq, tk = case["lq"], case["lk"]
            pairs = tq * (tq + 1) // 2 + tq * (tk - tq)
        B, Hq, Hkv, D = (case[k] for k in ("B", "Hq", "Hkv", "D"))
        return {"bytes": B * (2 * Hq * tq * D * e + 2 * Hkv * tk * D * e + 4 * Hq * tq), "flops": 4 * B * Hq * D * pairs}
    t, row = sum(lens), case["D"] // 2 + case["D"] // 32
    if op == "kv4_store":
        n = 2 * case["Hkv"] * t
        return {"bytes": 2 * n * (case["D"] * e + row), "flops": 4 * n * case["D"]}
    return {"bytes": 2 * case["Hkv"] * t * row + 2 * len(lens) * case["Hq"] * case["D"] * e, "flops": 4 * case["Hq"] * case["D"] * t}


# ---- in 64 bits, written apart ---------------------------------------------------------------------


def _padded(x, cu):
    """[1, H, T, d] packed -> [N, H, longest, d] in 64 bits, and which places hold tokens."""
    lens = [z - a for a, z in zip(cu, cu[1:])]
    out = torch.zeros(len(lens), x.shape[1], max(lens), x.shape[3], dtype=torch.float64, device=x.device)
    for n, (a, z) in enumerate(zip(cu, cu[1:])):
        out[n, :, :z - a] = x[0, :, a:z].double()
    return out


def _glr_exact(s, backward):
    """Token by token over all sequences at once, each laid out from its own first token."""
    cu = None if s["cu"] is None else s["cu_host"].tolist()
    g = s["g"].double() if cu is None else _padded(s["g"], cu)
    N, H, T, d = g.shape
    lens = torch.full((N,), T, device=g.device) if cu is None else torch.tensor(cu, device=g.device).diff()
    live = (torch.arange(T, device=g.device)[:, None] < lens[None]).double()[:, :, None, None]  # [T, N, 1, 1]

    def rows(x):
        if cu is None:
            return x
        return torch.cat([x[n, :, :z - a] for n, (a, z) in enumerate(zip(cu, cu[1:]))], 1)[None]

    if not backward:
        h = s["h0"].double()
        x = s["x"].double() if cu is None else _padded(s["x"], cu)
        out = torch.empty_like(x)
        for t in range(T):
            h = torch.lerp(h, torch.addcmul(x[:, :, t], g[:, :, t].exp(), h), live[t])
            out[:, :, t] = h
        return rows(out), h
    do, o = (s[k].double() if cu is None else _padded(s[k], cu) for k in ("do", "o"))
    dx, dg, carry = torch.empty_like(do), torch.empty_like(do), s["dfinal"].double()
    h0 = s["h0"].double()
    for t in range(T - 1, -1, -1):  # carry: the gradient that reaches the state behind token t
        dh = carry + do[:, :, t]
        back = g[:, :, t].exp() * dh
        dx[:, :, t], dg[:, :, t] = dh, back * (o[:, :, t - 1] if t else h0)
        carry = torch.lerp(carry, back, live[t])
    return rows(dx), rows(dg), carry


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("glr_fwd", "glr_bwd"):
        return _glr_exact(s, op == "glr_bwd")
    if op == "glr_step":
        h = torch.addcmul(s["x"].double(), s["g"].double().exp(), s["state"].double())
        return h, h
    if op == "attn":
        q, k, v = (s[n].double() for n in "qkv")
        off, group = k.shape[2] - q.shape[2], q.shape[1] // k.shape[1]
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:3], dtype=torch.float64, device=q.device)
        cu = [0, q.shape[2]] if s["cu"] is None else s["cu_host"].tolist()
        for b in range(q.shape[0]):
            for h in range(q.shape[1]):
                for a, z in zip(cu, cu[1:]):
                    for i in range(a, z, 2048):  # a run of queries against the keys it can see
                        w = min(i + 2048, z)
                        t = q[b, h, i:w] @ k[b, h // group, a:w + off].t() / math.sqrt(q.shape[3])
                        t = t.masked_fill(torch.ones_like(t, dtype=torch.bool).triu(i + off - a + 1), -math.inf)
                        lse[b, h, i:w] = torch.logsumexp(t, 1)
                        out[b, h, i:w] = (t - lse[b, h, i:w, None]).exp() @ v[b, h // group, a:w + off]
        return out, lse
    if op == "kv4_store":  # the nearest of the eight magnitudes, an even code where two are as near
        mags = torch.tensor(E2M1, dtype=torch.float64, device=s["k"].device)
        bias = torch.tensor([0.0, 1e-9] * 4, dtype=torch.float64, device=s["k"].device)
        both = []
        for x in (s["k"], s["v"]):
            b = x.double().unflatten(-1, (-1, 32))
            top = b.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -124)
            e = torch.exp2(torch.floor(torch.log2(top)) - 2)
            best, got = torch.full_like(b, math.inf), torch.zeros_like(b)
            for m, nudge in zip(mags, bias):
                far = ((b / e).abs() - m).abs() + nudge
                got = torch.where(far < best, m, got)
                best = torch.minimum(best, far)
            both.append((got * b.sign() * e).flatten(-2))
        return both
    D, Hkv = case["D"], case["Hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for n, L in enumerate(s["lens"].tolist()):
        pages = s["table"][n, : -(-L // PAGE)].long()
        for j in range(Hkv):
            k, v = (_values(s["codes"][pages, i, j], s["scales"][pages, i, j], torch.float64).reshape(-1, D)[:L] for i in (0, 1))
            rows = slice(j * (case["Hq"] // Hkv), (j + 1) * (case["Hq"] // Hkv))
            out[n, rows] = torch.softmax(s["q"][n, rows].double() @ k.t() / math.sqrt(D), -1) @ v
    return out
