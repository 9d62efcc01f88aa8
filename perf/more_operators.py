"""The measured cases of linear attention with a decay per head, and of what a 4-bit cache needs for
prompts that arrive in chunks and contexts that outgrow it: their inputs, their plain forms in
elementary torch operations, the calls of gated_delta_rule_kla_amd.kla that compute the same, and
what they give in 64 bits.

Operators (a case's "op"):
  la_fwd     S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t over packed or dense sequences
  la_bwd     its gradients for q, k, v, g and the initial state
  la_step    one token per sequence, the state updated in place
  kv4_chunk  causal softmax attention of each sequence's newest tokens over a 4-bit cache that
             holds them already, grouped heads; also the logarithm of each query's sum
  kv4_weigh  the attention weight that those tokens give to every cached token, summed over
             tokens and query heads and added to what earlier calls left
  kv4_evict  a cache cut to a budget: the newest tokens and, per key head, those of the largest
             weight stay in their order, in place; the kept values are read back

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
CHUNK = 64  # tokens that the plain form of linear attention takes at once


def listed():
    return [
        # a prefill of 4 x 4096 tokens through 16 heads of 128 x 128
        {"name": "la_fwd_prefill", "op": "la_fwd", "dt": "bf16", "B": 4, "H": 16, "T": 4096, "dk": 128, "dv": 128, "fixed": 0, "lo": 0, "pack": 0, "seqs": 0},
        # one long document, 65,536 tokens, with fixed decays: 16 heads and no other parallelism
        {"name": "la_fwd_long", "op": "la_fwd", "dt": "bf16", "B": 1, "H": 16, "T": 65536, "dk": 128, "dv": 256, "fixed": 1, "lo": 0, "pack": 0, "seqs": 0},
        # a training step's gradients over 16 packed documents of 256 to 8,192 tokens
        {"name": "la_bwd_packed", "op": "la_bwd", "dt": "bf16", "B": 1, "H": 16, "T": 0, "dk": 128, "dv": 128, "fixed": 0, "lo": 256, "pack": 8192, "seqs": 16},
        # the debug build's tiny fp32 shape: latency
        {"name": "la_bwd_tiny", "op": "la_bwd", "dt": "fp32", "B": 1, "H": 1, "T": 256, "dk": 16, "dv": 16, "fixed": 0, "lo": 0, "pack": 0, "seqs": 0},
        # one interactive user: a single token
        {"name": "la_step_one", "op": "la_step", "dt": "bf16", "N": 1, "H": 16, "dk": 128, "dv": 128, "fixed": 1},
        # a serving batch of 256 sequences
        {"name": "la_step_batch", "op": "la_step", "dt": "bf16", "N": 256, "H": 16, "dk": 128, "dv": 128, "fixed": 0},
        # 64 sequences whose five draft tokens are verified against up to 16,384 cached ones
        {"name": "kv4_chunk_verify", "op": "kv4_chunk", "dt": "bf16", "seqs": 64, "lo": 4096, "pack": 16384, "new": 5, "Hq": 16, "Hkv": 4, "D": 128},
        # a chunk of 2,048 tokens of one long prompt, 60,000 tokens into it
        {"name": "kv4_chunk_long", "op": "kv4_chunk", "dt": "bf16", "seqs": 1, "lo": 60000, "pack": 60000, "new": 2048, "Hq": 16, "Hkv": 2, "D": 128},
        # a serving batch's weights after each token
        {"name": "kv4_weigh_step", "op": "kv4_weigh", "dt": "bf16", "seqs": 64, "lo": 4096, "pack": 16384, "new": 1, "Hq": 16, "Hkv": 4, "D": 128},
        # the weights that chunks of up to 1,000 tokens of 12 prompts give
        {"name": "kv4_weigh_chunk", "op": "kv4_weigh", "dt": "bf16", "seqs": 12, "lo": 200, "pack": 4000, "new": 1000, "Hq": 16, "Hkv": 4, "D": 128},
        # a serving batch cut to 4,096 tokens a sequence
        {"name": "kv4_evict_batch", "op": "kv4_evict", "dt": "bf16", "seqs": 64, "lo": 4096, "pack": 16384, "budget": 4096, "recent": 256, "Hkv": 4, "D": 128},
        # one user's context of 131,071 tokens cut to 32,768
        {"name": "kv4_evict_long", "op": "kv4_evict", "dt": "bf16", "seqs": 1, "lo": 131071, "pack": 131071, "budget": 32768, "recent": 1000, "Hkv": 2, "D": 128},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["la_fwd", "la_bwd", "la_step", "kv4_chunk", "kv4_weigh", "kv4_evict"])
    dt = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("la_fwd", "la_bwd"):
        dk, dv = rng.choice([16, 48, 64, 128, 128, 256]), rng.choice([16, 64, 80, 128, 128, 256])
        H = rng.choice([1, 2, 5, 16])
        most = max(64, min(65536, (1 << (33 if op == "la_fwd" else 32)) // (H * max(dk, 64) * max(dv, 64))))  # tokens in all
        case = {"op": op, "dt": dt, "B": 1, "H": H, "T": 0, "dk": dk, "dv": dv, "fixed": rng.choice([0, 0, 1]) if op == "la_fwd" else 0, "lo": 0, "pack": 0, "seqs": 0}
        if rng.random() < 0.5:
            seqs = rng.randint(2, 24)
            top = max(8, min(8192, most // seqs))
            return {**case, "seqs": seqs, "lo": max(1, top // 32), "pack": _log_int(rng, max(2, top // 16), top)}
        B = rng.choice([1, 1, 3, 8])
        return {**case, "B": B, "T": _log_int(rng, 1, max(8, most // B))}
    if op == "la_step":
        return {"op": op, "dt": dt, "N": _log_int(rng, 1, 256), "H": rng.choice([1, 3, 16, 16]), "dk": rng.choice([16, 64, 128]), "dv": rng.choice([16, 48, 64, 128]), "fixed": rng.choice([0, 1])}
    Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    group = rng.choice([1, 2, 4, 5, 8])
    if op == "kv4_evict":
        seqs = _log_int(rng, 1, 64)
        top = _log_int(rng, 2, min(65536, 300000 // seqs))
        budget = _log_int(rng, 1, top)
        return {"op": op, "dt": dt, "seqs": seqs, "lo": max(1, top // 8), "pack": top, "budget": budget, "recent": rng.choice([0, rng.randint(0, budget), budget // 8]), "Hkv": Hkv, "D": D}
    new = rng.choice([1, rng.randint(2, 8), _log_int(rng, 8, 2000)])
    seqs = rng.choice([1, _log_int(rng, 1, 64)]) if new <= 8 else _log_int(rng, 1, 12)
    top = _log_int(rng, 1, min(60000, 300000 // seqs if new <= 8 else 60000 // seqs))
    new = min(new, max(8, 1500000000 // (Hkv * group * seqs * (top + new))))
    return {"op": op, "dt": dt, "seqs": seqs, "lo": max(1, top // 8), "pack": top, "new": new, "Hq": Hkv * group, "Hkv": Hkv, "D": D}


def _lengths(case, lo, pack):
    """The case's own ragged lengths, log-uniform in [lo, pack]; they do not depend on the seed."""
    rng = random.Random(case["seqs"] * 1000003 + lo * 1009 + pack)
    return [_log_int(rng, lo, pack) if pack > lo else lo for _ in range(case["seqs"])]


def _tokens(case):
    """Per sequence of a kv4 case: its new tokens and its cached ones, the new among them."""
    before = _lengths(case, case["lo"], case["pack"])
    new = [case["new"]] * case["seqs"] if case["new"] <= 8 or case["seqs"] == 1 else _lengths(case, max(1, case["new"] // 8), case["new"])
    return new, [a + b for a, b in zip(new, before)]


def _bounds(lens, dev):
    host = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
    return host.to(dev), host


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, op = DT[case["dt"]], case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(std)

    s = {"case": case}
    if op.startswith("la_"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        # heads remember from a few tokens to some thousands
        rate = torch.exp2(-torch.linspace(1, 11, H, device=dev))
        if op == "la_step":
            N, lead = case["N"], (case["N"], H)
        else:
            B, T = case["B"], case["T"]
            N, s["cu"], s["cu_host"] = B, None, None
            if case["seqs"]:
                lens = _lengths(case, case["lo"], case["pack"])
                N, T = len(lens), sum(lens)
                s["cu"], s["cu_host"] = _bounds(lens, dev)
            lead = (B, H, T)
        s["q"], s["k"], s["v"] = normal(*lead, dk, std=dk ** -0.5).to(dt), normal(*lead, dk, std=dk ** -0.5).to(dt), normal(*lead, dv).to(dt)
        if case["fixed"]:
            s["g"] = -rate
        else:
            s["g"] = (torch.nn.functional.softplus(normal(*lead)) * -(rate if op == "la_step" else rate[:, None])).to(dt)
        if op == "la_step":
            s["state"] = normal(N, H, dk, dv)
        else:
            s["h0"] = normal(N, H, dk, dv)
        if op == "la_bwd":
            s["do"], s["dfinal"] = normal(*lead, dv).to(dt), normal(N, H, dk, dv)
        return s
    Hkv, D = case["Hkv"], case["D"]
    new, lens = ([], _lengths(case, case["lo"], case["pack"])) if op == "kv4_evict" else _tokens(case)
    M = -(-max(lens) // PAGE)
    P = len(lens) * M + 3
    order = torch.randperm(P, generator=gen, device=dev)[: len(lens) * M]
    s["table"] = order.to(torch.int32).reshape(len(lens), M).contiguous()
    s["codes"] = torch.zeros(P, 2, Hkv, PAGE, D // 2, dtype=torch.uint8, device=dev)
    s["scales"] = torch.zeros(P, 2, Hkv, PAGE, D // 32, dtype=torch.uint8, device=dev)
    loud = 1 + 3 * (torch.rand(Hkv, 1, D, generator=gen, device=dev) < 0.03)  # a few channels of keys are large
    for p in range(0, P, 512):
        n = min(512, P - p)
        for j, m in ((0, loud), (1, 1.0)):
            s["codes"][p:p + n, j], s["scales"][p:p + n, j] = _quantise((normal(n, Hkv, PAGE, D) * m).to(torch.bfloat16).float())
    s["lens"], s["max_len"] = torch.tensor(lens, dtype=torch.int32, device=dev), max(lens)
    # weights as many steps of attention leave them: a few tokens hold most, some none at all
    w = torch.exp(normal(len(lens), Hkv, M * PAGE, std=2.0)) * (torch.rand(len(lens), Hkv, M * PAGE, generator=gen, device=dev) > 0.05)
    s["weights"] = w.masked_fill_(torch.arange(M * PAGE, device=dev) >= s["lens"][:, None, None], 0.0)
    if op == "kv4_evict":
        s["zero"] = torch.zeros_like(s["lens"])
        s["kept_cu"], s["kept_host"] = _bounds([min(n, case["budget"]) for n in lens], dev)
        return s
    s["q"] = normal(1, case["Hq"], sum(new), D).to(dt)
    s["cu"], s["cu_host"] = _bounds(new, dev)
    if op == "kv4_weigh":
        s["lse"] = _kv4_chunk(s, values=False)
    return s


# ---- the plain forms -------------------------------------------------------------------------


def _chunks(s, C=CHUNK):
    """Linear attention's tokens in chunks that cross no sequence: indexes [chunks, C] into the
    tokens of all batch rows, which of them are tokens, each chunk's sequence, and each
    sequence's first and last chunk."""
    B, _, T, _ = s["q"].shape
    dev = s["q"].device
    if s["cu"] is None:
        first = torch.arange(B, device=dev) * T
        n = torch.full_like(first, T)
        count = B * -(-T // C)
    else:
        first, n = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
        count = int((-(-s["cu_host"].diff() // C)).sum())
    per = -(-n // C)
    end = per.cumsum(0)
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=dev), per, output_size=count)
    at = (torch.arange(count, device=dev) - (end - per)[seq])[:, None] * C + torch.arange(C, device=dev)
    there = at < n[seq][:, None]
    return (first[seq][:, None] + at).where(there, first[seq][:, None]), there, seq, end - per, end - 1


def _laid_out(x, idx, there):
    """[B, H, T, ...] -> [H, chunks, C, ...], zero where there is no token."""
    y = x.transpose(0, 1).flatten(1, 2)[:, idx]
    return y.masked_fill(~there.view(there.shape + (1,) * (x.dim() - 3)), 0.0)


def _put_back(y, like, idx, there):
    B, H, T = like.shape[:3]
    out = torch.empty((H, B * T) + tuple(y.shape[3:]), dtype=like.dtype, device=like.device)
    out[:, idx[there]] = y[:, there].to(like.dtype)
    return out.unflatten(1, (B, T)).transpose(0, 1).contiguous()


def _scan(a, U):
    """S_c = a_c S_{c-1} + U_c along dim 1 by doubling; a [H, chunks], U [H, chunks, dk, dv]."""
    step, n = 1, a.shape[1]
    a, U = a[..., None, None].clone(), U.clone()
    while step < n:
        U[:, step:] = U[:, step:] + a[:, step:] * U[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    return U


def _la(s):
    """What the forward and backward share: chunks, decays and the state at each chunk's start."""
    idx, there, seq, first, last = _chunks(s)
    g = s["g"] if s["g"].dim() == 3 else s["g"][None, :, None].expand(s["q"].shape[:3])
    q, k, v = (_laid_out(s[n].float(), idx, there) for n in "qkv")
    cum = _laid_out(g.double(), idx, there).cumsum(2)
    tot = cum[:, :, -1:]
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    D = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~tri, -math.inf)).float()
    out, left = torch.exp(cum).float()[..., None], torch.exp(tot - cum).float()[..., None]
    a = torch.exp(tot[:, :, 0]).float()
    h0 = s["h0"].transpose(0, 1)
    U, b = (k * left).transpose(2, 3) @ v, a.clone()
    U[:, first] += a[:, first, None, None] * h0
    b[:, first] = 0.0
    ends = _scan(b, U)
    S = torch.cat((ends[:, :1], ends[:, :-1]), 1)
    S[:, first] = h0
    return idx, there, first, last, q, k, v, D, out, left, a, S, ends


def _la_fwd(s):
    idx, there, first, last, q, k, v, D, out, left, a, S, ends = _la(s)
    o = ((q @ k.transpose(2, 3)) * D) @ v + out * (q @ S)
    return _put_back(o, s["v"], idx, there), ends[:, last].transpose(0, 1).contiguous()


def _la_bwd(s):
    idx, there, first, last, q, k, v, D, out, left, a, S, ends = _la(s)
    do, df = _laid_out(s["do"].float(), idx, there), s["dfinal"].transpose(0, 1)
    U, b = (q * out).transpose(2, 3) @ do, a.clone()
    U[:, last] += a[:, last, None, None] * df
    b[:, last] = 0.0
    back = _scan(b.flip(1), U.flip(1)).flip(1)  # the gradient that reaches each chunk's start state
    M = torch.cat((back[:, 1:], back[:, -1:]), 1)  # and its end state
    M[:, last] = df
    P, dP = (q @ k.transpose(2, 3)) * D, (do @ v.transpose(2, 3)) * D
    qi, ki = out * (do @ S.transpose(2, 3)), left * (v @ M.transpose(2, 3))
    dq, dk = dP @ k + qi, dP.transpose(2, 3) @ q + ki
    dv = P.transpose(2, 3) @ do + left * (k @ M)
    # the decay of token t stands between every write before t and every read from t on
    W = (P * (do @ v.transpose(2, 3))).tril(-1)
    reads, writes = (q * qi).sum(3), (k * ki).sum(3)
    ahead = W.sum(3) - W.sum(2) + reads
    dg = ahead.flip(2).cumsum(2).flip(2) + writes.cumsum(2) - writes + (a * (M * S).sum((2, 3)))[..., None]
    return (_put_back(dq, s["q"], idx, there), _put_back(dk, s["k"], idx, there), _put_back(dv, s["v"], idx, there),
            _put_back(dg, s["g"], idx, there), back[:, first].transpose(0, 1).contiguous())


def _la_step(s):
    g = s["g"].float()[..., None, None]
    s["state"].copy_(torch.exp(g) * s["state"] + s["k"].float()[..., None] * s["v"].float()[..., None, :])
    return (s["q"].float()[..., None] * s["state"]).sum(2).to(s["q"].dtype), s["state"]


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


def _cached(s, n, L, j, h):
    """Keys (j = 0) or values (j = 1) of sequence n's first L tokens for a head, in fp32."""
    pages = s["table"][n, : -(-L // PAGE)].long()
    return _values(s["codes"][pages, j, h], s["scales"][pages, j, h]).flatten(0, 1)[:L]


def _spans(s):
    """Each sequence with its queries' range, its cached tokens, and a key head with its queries'."""
    new, lens = _tokens(s["case"])
    group, cu = s["q"].shape[1] // s["codes"].shape[2], s["cu_host"].tolist()
    for n, L in enumerate(lens):
        for h in range(s["codes"].shape[2]):
            yield n, cu[n], cu[n + 1], L, h, slice(h * group, (h + 1) * group)


def _kv4_chunk(s, values=True):
    q = s["q"]
    D = q.shape[3]
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    for n, a, z, L, h, rows in _spans(s):
        k = _cached(s, n, L, 0, h).T.contiguous()
        v = _cached(s, n, L, 1, h) if values else None
        sc = q[0, rows, a:z].float() @ k * D ** -0.5
        ends = torch.arange(L - (z - a), L, device=q.device)[:, None]
        sc.masked_fill_(torch.arange(L, device=q.device)[None, :] > ends, -math.inf)
        top = sc.amax(2, keepdim=True)
        p = sc.sub_(top).exp_()
        tot = p.sum(2, keepdim=True)
        lse[0, rows, a:z] = (top + torch.log(tot))[..., 0]
        if values:
            out[0, rows, a:z] = ((p @ v) / tot).to(q.dtype)
    return (out, lse) if values else lse


def _kv4_weigh(s):
    q = s["q"]
    D = q.shape[3]
    for n, a, z, L, h, rows in _spans(s):
        sc = q[0, rows, a:z].float() @ _cached(s, n, L, 0, h).T.contiguous() * D ** -0.5
        ends = torch.arange(L - (z - a), L, device=q.device)[:, None]
        sc.masked_fill_(torch.arange(L, device=q.device)[None, :] > ends, -math.inf)
        s["weights"][n, h, :L] += sc.sub_(s["lse"][0, rows, a:z, None]).exp_().sum((0, 1))
    return s["weights"]


def _rows(s, pos):
    """Page and place in it of positions pos [N, Hkv, n] of the cache."""
    n = torch.arange(pos.shape[0], device=pos.device)[:, None, None]
    return s["table"][n, pos // PAGE].long(), pos % PAGE


def _kv4_evict(s):
    case, w = s["case"], s["weights"]
    budget, dev = case["budget"], w.device
    lens, pos = s["lens"].long()[:, None, None], torch.arange(w.shape[2], device=dev)
    order = w.masked_fill(pos >= lens, -math.inf).masked_fill((pos >= lens - case["recent"]) & (pos < lens), math.inf)
    order = torch.sort(order, dim=2, descending=True, stable=True).indices[..., :budget]
    src = torch.sort(order, dim=2).values
    to = torch.arange(src.shape[2], device=dev)
    live = to < lens.clamp(max=budget)
    src = torch.where(live, src, to)
    h = torch.arange(w.shape[1], device=dev)[:, None]
    (p0, a0), (p1, a1) = _rows(s, src), _rows(s, to.expand_as(src))
    for j in (0, 1):
        for x in (s["codes"], s["scales"]):
            x[p1, j, h, a1] = x[p0, j, h, a0]
    moved = torch.gather(w, 2, src)
    over = (pos >= budget) & (pos < lens)
    w.masked_fill_(over, 0.0)
    w[..., :src.shape[2]] = torch.where(live, moved, w[..., :src.shape[2]])
    kept = torch.full((w.shape[0], w.shape[1], budget), -1, dtype=torch.int32, device=dev)
    kept[..., :src.shape[2]] = torch.where(live, src, -1).to(torch.int32)
    both = []
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device=dev), s["kept_cu"].diff().long(), output_size=int(s["kept_host"][-1]))
    at = torch.arange(seq.numel(), device=dev) - s["kept_cu"].long()[seq]
    page = s["table"][seq, at // PAGE].long()
    for j in (0, 1):
        x = _values(s["codes"][page, j, :, at % PAGE], s["scales"][page, j, :, at % PAGE])
        both.append(x.transpose(0, 1).to(DT[case["dt"]]).contiguous()[None])
    return {"lens": s["lens"].clamp(max=budget), "kept": kept, "weights": w, "k": both[0], "v": both[1]}


PLAIN = {"la_fwd": _la_fwd, "la_bwd": _la_bwd, "la_step": _la_step, "kv4_chunk": _kv4_chunk, "kv4_weigh": _kv4_weigh,
         "kv4_evict": _kv4_evict}


# ---- the framework's calls ---------------------------------------------------------------------


def _calls(s):
    from gated_delta_rule_kla_amd import kla

    case = s["case"]
    op = case["op"]
    if op == "la_fwd":
        return kla.la_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], s["cu"], cu_seqlens_host=s["cu_host"])
    if op == "la_bwd":
        return kla.la_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], s["h0"], s["dfinal"], s["cu"], cu_seqlens_host=s["cu_host"])
    if op == "la_step":
        return kla.la_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"]), s["state"]
    if op == "kv4_chunk":
        return kla.attn_kv4_chunk_fwd(s["q"], s["codes"], s["scales"], s["table"], s["lens"], s["cu"], cu_seqlens_host=s["cu_host"], max_len=s["max_len"])
    if op == "kv4_weigh":
        kla.attn_kv4_weigh(s["q"], s["lse"], s["codes"], s["scales"], s["table"], s["lens"], s["weights"], s["cu"], cu_seqlens_host=s["cu_host"], max_len=s["max_len"])
        return s["weights"]
    lens, kept = kla.kv4_evict(s["codes"], s["scales"], s["table"], s["lens"], s["weights"], case["budget"], case["recent"])
    k, v = kla.kv4_read(s["codes"], s["scales"], s["table"], s["zero"], s["kept_cu"], DT[case["dt"]], cu_seqlens_host=s["kept_host"])
    return {"lens": lens, "kept": kept, "weights": s["weights"], "k": k, "v": v}


def run(s):
    return _calls(s) if own else PLAIN[s["case"]["op"]](s)


# ---- what a pass cannot do without -----------------------------------------------------------------


def work(case):
    op, e = case["op"], 2 if case["dt"] == "bf16" else 4
    if op.startswith("la_"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        if op == "la_step":
            n = case["N"] * H
            return {"bytes": n * ((2 * dk + 2 * dv) * e + 8 * dk * dv), "flops": 5 * n * dk * dv}
        lens = _lengths(case, case["lo"], case["pack"]) if case["seqs"] else [case["T"]] * case["B"]
        n, states = H * sum(lens), H * len(lens) * dk * dv * 4
        # token by token: the state's update and its reading, and the same again for each gradient
        if op == "la_fwd":
            return {"bytes": n * ((2 * dk + 2 * dv) * e + (0 if case["fixed"] else e)) + 2 * states, "flops": 4 * n * dk * dv}
        return {"bytes": n * ((4 * dk + 3 * dv) * e + 2 * e) + 3 * states, "flops": 10 * n * dk * dv}
    Hkv, D = case["Hkv"], case["D"]
    row = D // 2 + D // 32
    if op == "kv4_evict":
        lens = _lengths(case, case["lo"], case["pack"])
        kept = [min(n, case["budget"]) for n in lens]
        moved = sum(b for n, b in zip(lens, kept) if n > b)
        # weights read; kept rows, weights and positions written; the kept values read back
        return {"bytes": Hkv * (4 * sum(lens) + moved * (4 * row + 4) + 4 * case["seqs"] * case["budget"] + 2 * sum(kept) * (row + D * e)), "flops": Hkv * sum(lens)}
    new, lens = _tokens(case)
    pairs = sum(a * n - a * (a - 1) // 2 for a, n in zip(new, lens))
    q = case["Hq"] * sum(new)
    if op == "kv4_chunk":
        return {"bytes": 2 * Hkv * sum(lens) * row + 2 * q * D * e + 4 * q, "flops": 4 * case["Hq"] * D * pairs}
    return {"bytes": Hkv * sum(lens) * (row + 8) + q * D * e + 4 * q, "flops": 2 * case["Hq"] * D * pairs}


# ---- in 64 bits, written apart ---------------------------------------------------------------------


def _padded(x, cu):
    """[1, H, T, ...] packed -> [N, H, longest, ...] in 64 bits."""
    if cu is None:
        return x.double()
    out = x.new_zeros((len(cu) - 1, x.shape[1], max(z - a for a, z in zip(cu, cu[1:]))) + tuple(x.shape[3:]), dtype=torch.float64)
    for n, (a, z) in enumerate(zip(cu, cu[1:])):
        out[n, :, :z - a] = x[0, :, a:z].double()
    return out


def _la_exact(s, backward):
    """Token by token over all sequences at once, each laid out from its own first token."""
    cu = None if s["cu"] is None else s["cu_host"].tolist()
    q, k, v = (_padded(s[n], cu) for n in "qkv")
    N, H, T, dk = q.shape
    dev = q.device
    lens = torch.full((N,), T, device=dev) if cu is None else torch.tensor(cu, device=dev).diff()
    live = (torch.arange(T, device=dev)[:, None] < lens[None]).double()[:, :, None, None, None]  # [T, N, 1, 1, 1]
    g = _padded(s["g"], cu) if s["g"].dim() == 3 else s["g"].double()[None, :, None].expand(N, H, T)
    # behind a sequence's end: no write and no decay
    f = torch.exp(g * live[..., 0, 0].permute(1, 2, 0))[..., None, None]

    def rows(x):
        if cu is None:
            return x
        return torch.cat([x[n, :, :z - a] for n, (a, z) in enumerate(zip(cu, cu[1:]))], 1)[None]

    S, kt = s["h0"].double(), k[..., None]
    o = torch.empty_like(v)
    if not backward:
        for t in range(T):
            S = torch.baddbmm((S * f[:, :, t]).flatten(0, 1), kt[:, :, t].flatten(0, 1), v[:, :, t, None].flatten(0, 1)).unflatten(0, (N, H))
            o[:, :, t] = (q[:, :, t, None] @ S)[:, :, 0]
        return rows(o), S
    do = _padded(s["do"], cu)
    dq, dkk, dvv, dG = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(g)
    for t in range(T):
        S = torch.baddbmm((S * f[:, :, t]).flatten(0, 1), kt[:, :, t].flatten(0, 1), v[:, :, t, None].flatten(0, 1)).unflatten(0, (N, H))
        dq[:, :, t] = (S @ do[:, :, t, :, None])[..., 0]
    M = s["dfinal"].double()
    end = (M * S).sum((2, 3))
    for t in range(T - 1, -1, -1):  # M: the gradient that reaches the state behind token t
        M = M + q[:, :, t, :, None] * do[:, :, t, None]
        dkk[:, :, t] = (M @ v[:, :, t, :, None])[..., 0]
        dvv[:, :, t] = (k[:, :, t, None] @ M)[:, :, 0]
        M = M * f[:, :, t]
    # what a token's decay changes: all reads from it on, less the writes from it on
    dG = (q * dq).sum(3) - (k * dkk).sum(3)
    dg = dG.flip(2).cumsum(2).flip(2) + end[..., None]
    return rows(dq), rows(dkk), rows(dvv), rows(dg), M


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("la_fwd", "la_bwd"):
        return _la_exact(s, op == "la_bwd")
    if op == "la_step":
        f = s["g"].double().exp().reshape(-1, case["H"], 1, 1)
        S = torch.einsum("nhk,nhv->nhkv", s["k"].double(), s["v"].double()) + f * s["state"].double()
        return torch.einsum("nhk,nhkv->nhv", s["q"].double(), S), S
    if op == "kv4_evict":  # each head by itself, its kept values taken before anything moves
        w, rows = s["weights"].double().cpu().numpy(), [[], []]
        for n, L in enumerate(s["lens"].tolist()):
            pages, took = s["table"][n, : -(-L // PAGE)].long(), [[], []]
            for h in range(case["Hkv"]):
                free = L - min(case["recent"], L)
                keep = np.arange(L)
                if L > case["budget"]:
                    best = np.lexsort((keep[:free], -w[n, h, :free]))[: case["budget"] - case["recent"]]
                    keep = np.concatenate((np.sort(best), keep[free:]))
                w[n, h, :L] = np.concatenate((w[n, h, keep], np.zeros(L - keep.size)))
                for i in (0, 1):
                    took[i].append(_values(s["codes"][pages, i, h], s["scales"][pages, i, h], torch.float64).flatten(0, 1)[torch.from_numpy(keep).to(pages.device)])
            for i in (0, 1):
                rows[i].append(torch.stack(took[i]))
        return {"lens": None, "kept": None, "weights": torch.from_numpy(w), "k": torch.cat(rows[0], 1)[None], "v": torch.cat(rows[1], 1)[None]}
    q, D, Hkv = s["q"][0].double(), case["D"], case["Hkv"]
    group = case["Hq"] // Hkv
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    weights = s["weights"].double()
    new, lens = _tokens(case)
    a = 0
    for n, (m, L) in enumerate(zip(new, lens)):
        pages = s["table"][n, : -(-L // PAGE)].long()
        for h in range(case["Hq"]):
            k, v = (_values(s["codes"][pages, i, h // group], s["scales"][pages, i, h // group], torch.float64).reshape(-1, D)[:L] for i in (0, 1))
            for i in range(0, m, 1024):  # a run of queries against the keys it can see
                w = min(i + 1024, m)
                seen = L - m + w
                t = q[h, a + i:a + w] @ k[:seen].t() / math.sqrt(D)
                t = t.masked_fill(torch.ones_like(t, dtype=torch.bool).triu(seen - (w - i) + 1), -math.inf)
                if op == "kv4_weigh":
                    weights[n, h // group, :seen] += (t - s["lse"][0, h, a + i:a + w, None].double()).exp().sum(0)
                else:
                    lse[h, a + i:a + w] = torch.logsumexp(t, 1)
                    out[h, a + i:a + w] = (t - lse[h, a + i:a + w, None]).exp() @ v[:seen]
        a += m
    return weights if op == "kv4_weigh" else (out[None], lse[None])
