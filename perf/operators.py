"""Measured cases of the multi-token MLA operators: appending rows to the paged latent cache with
the position rotation, causal attention over whole packed prompts, and attention of a chunk of
new tokens over the paged latent cache.

`run` computes each operator in elementary torch operations (32 bits, 64 for the angles), or,
where `own` is true, through the package's calls.  `exact` gives the same outputs in 64 bits.

Sizes: n_heads 16 ... 128 in steps of 16 (the head counts the package takes), 64-token pages,
latent rows of 512 + 64, head widths 128 + 64 (query, key) and 128 (value).
"""
import math

import torch

own = False

D_C, D_R, D_N, D_V, PAGE = 512, 64, 128, 128, 64
ROW, D_QK = D_C + D_R, D_N + D_R
SCALE = 1.0 / math.sqrt(D_QK)
THETA = 10000.0


def _ints(text):
    return [int(x) for x in text.split(",")]


def listed():
    return [
        # one new token for each of 16 sequences: the cache write of a small decode step
        dict(name="append_single", op="append", dtype="bf16", heads=128,
             tokens=",".join(["1"] * 16), lens=",".join(str(900 + 211 * i) for i in range(16))),
        # chunks of prompts of several lengths entering the cache in one call
        dict(name="append_chunk", op="append", dtype="bf16", heads=128,
             tokens="2048,1,511,4096,65,1000,300,171", lens="2048,4097,1023,8192,65,9000,811,6000"),
        # the 32-bit configuration
        dict(name="append_f32", op="append", dtype="f32", heads=16, tokens="700,300,24",
             lens="700,1300,131071"),
        # a few short requests: latency
        dict(name="prompt_short", op="prompt", dtype="bf16", heads=16, kv_heads=16,
             tokens="65,17,1,130"),
        # a batch of prompts as a server packs them, every head with keys of its own
        dict(name="prompt_packed", op="prompt", dtype="bf16", heads=128, kv_heads=128,
             tokens="4096,2048,1000,700,300,48"),
        # one long document, eight query heads to a key head
        dict(name="prompt_long", op="prompt", dtype="bf16", heads=32, kv_heads=4, tokens="16384"),
        # the 32-bit configuration, grouped heads
        dict(name="prompt_f32", op="prompt", dtype="f32", heads=16, kv_heads=4,
             tokens="500,129,33"),
        # one token for each of eight sequences: the smallest call
        dict(name="chunk_single", op="chunk", dtype="bf16", heads=128, tokens="1,1,1,1,1,1,1,1",
             lens="1024,2048,1500,3000,700,64,1,2500"),
        # a few proposed tokens for each of 32 sequences, verified in one pass
        dict(name="chunk_verify", op="chunk", dtype="bf16", heads=128,
             tokens=",".join(["4"] * 32), lens=",".join(str(4096 + 130 * i) for i in range(32))),
        # one prompt chunk that shares the step with sequences that decode
        dict(name="chunk_mixed", op="chunk", dtype="bf16", heads=128,
             tokens="512," + ",".join(["1"] * 24),
             lens="8192," + ",".join(str(300 + 331 * i) for i in range(24))),
        # a chunk of a long prompt over its cached beginning
        dict(name="chunk_prefill", op="chunk", dtype="bf16", heads=128, tokens="1024",
             lens="16384"),
        # the 32-bit configuration
        dict(name="chunk_f32", op="chunk", dtype="f32", heads=16, tokens="33,7", lens="700,129"),
    ]


def _log_int(rng, lo, hi):
    """An integer of lo ... hi, uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("append", "prompt", "chunk"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    heads = 16 * rng.randint(1, 8)
    case = dict(op=op, dtype=dtype, heads=heads)
    if op == "append":
        n = _log_int(rng, 1, 32)
        room = 8000 * 128 // heads if dtype == "bf16" else 2000
        tokens = [_log_int(rng, 1, max(1, min(4096, room // n))) for _ in range(n)]
        lens = [t + rng.randint(0, 1) * _log_int(rng, 1, 4000) for t in tokens]
    elif op == "prompt":
        case["kv_heads"] = heads // rng.choice([g for g in (1, 2, 4, 8, 16) if heads % g == 0])
        n = _log_int(rng, 1, 16)
        # every score of a sequence at most as many as in the longest listed prompt's share
        room = 2.0e9 if dtype == "bf16" else 4.0e7
        tokens = [_log_int(rng, 1, max(1, int(math.sqrt(room / heads / n)))) for _ in range(n)]
        lens = []
    else:
        n = _log_int(rng, 1, 32)
        room = 1.5e9 if dtype == "bf16" else 2.0e7
        lens, tokens = [], []
        for _ in range(n):
            length = _log_int(rng, 1, 16384 if dtype == "bf16" else 2000)
            most = max(1, min(length, 1024, int(room / heads / n / length)))
            lens.append(length)
            tokens.append(_log_int(rng, 1, most))
    case["tokens"] = ",".join(map(str, tokens))
    if lens:
        case["lens"] = ",".join(map(str, lens))
    return case


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    H, tokens = case["heads"], _ints(case["tokens"])
    T, B = sum(tokens), len(tokens)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case=case, T=T, H=H, dt=dt, n=tokens)
    s["cu"] = torch.tensor([sum(tokens[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
    if case["op"] == "prompt":
        Hk = case["kv_heads"]
        s["q"] = randn(T, H, D_QK).to(dt)
        # the up-projection writes keys and values of a head side by side; both are views of it
        kv = randn(T, Hk, D_N + D_V).to(dt)
        s["k_nope"], s["v"] = kv[..., :D_N], kv[..., D_N:]
        s["k_rope"] = randn(T, D_R).to(dt)
        s["o"] = torch.empty(T, H, D_V, dtype=dt, device=dev)
        s["lse"] = torch.empty(T, H, dtype=torch.float32, device=dev)
        return s
    lens = _ints(case["lens"])
    pages = [-(-n // PAGE) for n in lens]
    perm = torch.randperm(sum(pages), generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32, device=dev)
    for b in range(B):
        table[b, :pages[b]] = perm[sum(pages[:b]):sum(pages[:b + 1])]
    s["lens_host"], s["table"] = lens, table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["pool"] = randn(sum(pages), PAGE, ROW).to(dt)
    if case["op"] == "append":
        s["c_kv"], s["k_r"] = randn(T, D_C).to(dt), randn(T, D_R).to(dt)
        s["q"] = randn(T, H, D_QK).to(dt)
        s["q_cat"] = torch.empty(T, H, ROW, dtype=dt, device=dev)
        s["k_rope"] = torch.empty(T, D_R, dtype=dt, device=dev)
    else:
        q = randn(T, H, ROW)
        q[..., :D_C] *= 0.5
        s["q_cat"] = q.to(dt)
        s["o"] = torch.empty(T, H, D_C, dtype=dt, device=dev)
        s["lse"] = torch.empty(T, H, dtype=torch.float32, device=dev)
    return s


# --------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------
def _rotate(x, cos, sin):
    """Pairs (x[2i], x[2i+1]) turned by their angle; 32 bits, rounded by the caller."""
    x = x.float()
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack((x0 * cos - x1 * sin, x0 * sin + x1 * cos), -1).flatten(-2)


def _append(s):
    cu, lens, dev = s["cu"].long(), s["lens"].long(), s["cu"].device
    t = torch.arange(s["T"], device=dev)
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = lens[b] - cu[b + 1] + t
    freq = THETA ** (-torch.arange(0, D_R, 2, device=dev, dtype=torch.float64) / D_R)
    ang = pos.double()[:, None] * freq
    cos, sin = ang.cos().float(), ang.sin().float()
    k = _rotate(s["k_r"], cos, sin).to(s["dt"])
    s["pool"][s["table"][b, pos // PAGE].long(), pos % PAGE] = torch.cat((s["c_kv"], k), 1)
    s["k_rope"].copy_(k)
    s["q_cat"][..., D_C:] = _rotate(s["q"][..., D_N:], cos[:, None], sin[:, None]).to(s["dt"])
    return {"pool": s["pool"], "k_rope": s["k_rope"], "q_rope": s["q_cat"][..., D_C:]}


def _softmax_products(scores, hidden, v):
    """softmax over the last axis with the hidden places left out, times v, and the logarithm of
    the sum; the scores' memory is used again."""
    scores.mul_(SCALE).masked_fill_(hidden, -math.inf)
    m = scores.amax(-1, keepdim=True)
    e = scores.sub_(m).exp_()
    tot = e.sum(-1, keepdim=True)
    return (e @ v).div_(tot), (m + tot.log()).squeeze(-1)


def _prompt(s):
    o, lse, at, H = [], [], 0, s["H"]
    for n in s["n"]:  # the packed prompts are problems of their own
        q = s["q"][at:at + n].float().transpose(0, 1)
        k_nope = s["k_nope"][at:at + n].float().transpose(0, 1)
        Hk = k_nope.shape[0]
        k_rope = s["k_rope"][at:at + n].float().expand(Hk, n, D_R)
        k, v = torch.cat((k_nope, k_rope), -1), s["v"][at:at + n].float().transpose(0, 1)
        i = torch.arange(n, device=q.device)
        hidden = (i[None, :] > i[:, None]).repeat(H // Hk, 1)  # rows: heads of a group, tokens
        a, b = _softmax_products(q.reshape(Hk, H // Hk * n, D_QK) @ k.transpose(1, 2), hidden, v)
        o.append(a.reshape(H, n, D_V).transpose(0, 1))
        lse.append(b.reshape(H, n).t())
        at += n
    return {"o": torch.cat(o).to(s["dt"]), "lse": torch.cat(lse)}


def _chunk(s):
    n, lens, H, dev = s["n"], s["lens_host"], s["H"], s["cu"].device
    B = len(n)
    o = torch.empty(s["T"], H, D_C, device=dev)
    lse = torch.empty(s["T"], H, device=dev)
    # all sequences as one padded batch where that at most doubles the work, else one by one
    padded = B * max(n) * max(lens) <= 2 * sum(x * y for x, y in zip(n, lens))
    for group in [list(range(B))] if padded else [[b] for b in range(B)]:
        G, n_g, len_g = len(group), max(n[b] for b in group), max(lens[b] for b in group)
        first, last = group[0], group[-1] + 1
        cu, cnt = s["cu"][first:last].long(), (s["cu"][first + 1:last + 1] - s["cu"][first:last])
        pages = s["table"][first:last, :-(-len_g // PAGE)].clamp(min=0).long()
        rows = s["pool"][pages].reshape(G, -1, ROW)[:, :len_g].float()
        i, j = torch.arange(n_g, device=dev), torch.arange(len_g, device=dev)
        there = i[None, :] < cnt[:, None]
        t = (cu[:, None] + i).clamp(max=s["T"] - 1)
        q = s["q_cat"][t].float().reshape(G, n_g * H, ROW)
        pos = s["lens"][first:last, None] - cnt[:, None] + i
        hidden = (j > pos[..., None]).repeat_interleave(H, 1)
        a, b = _softmax_products(q @ rows.transpose(1, 2), hidden, rows[..., :D_C])
        o[t[there]] = a.reshape(G, n_g, H, D_C)[there]
        lse[t[there]] = b.reshape(G, n_g, H)[there]
    return {"o": o.to(s["dt"]), "lse": lse}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _append, "prompt": _prompt, "chunk": _chunk}[op](s)
    import mla_latent_kv_37_b200 as M
    if "dims" not in s:
        s["dims"] = M.dims(len(s["n"]), s["H"], dtype=s["dt"])
        if op == "chunk":
            s["ws"] = M.chunk_workspace(s["dims"], s["T"])
    d = s["dims"]
    if op == "append":
        q_out = s["q_cat"][..., D_C:]
        M.mla_append_rows(d, s["c_kv"], s["k_r"], s["cu"], s["lens"], s["table"], s["pool"],
                          k_rope=s["k_rope"], q_rope=s["q"][..., D_N:], q_rope_out=q_out)
        return {"pool": s["pool"], "k_rope": s["k_rope"], "q_rope": q_out}
    if op == "prompt":
        M.mla_prompt_attn(d, s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu"], s["o"],
                          lse=s["lse"])
    else:
        M.mla_chunk_attn(d, s["q_cat"], s["pool"], s["table"], s["cu"], s["lens"], s["o"],
                         s["ws"], lse=s["lse"])
    return {"o": s["o"], "lse": s["lse"]}


# --------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    H, tokens = case["heads"], _ints(case["tokens"])
    T = sum(tokens)
    if case["op"] == "append":
        moved = T * (2 * ROW + D_R + 2 * H * D_R) * e  # rows in and out, k_rope out, q in and out
        return {"bytes": moved, "flops": T * (H + 1) * D_R // 2 * 6}
    if case["op"] == "prompt":
        pairs = sum(n * (n + 1) // 2 for n in tokens)
        moved = T * (H * (D_QK + D_V) + case["kv_heads"] * (D_N + D_V) + D_R) * e + T * H * 4
        return {"bytes": moved, "flops": 2 * pairs * H * (D_QK + D_V)}
    lens = _ints(case["lens"])
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(tokens, lens))
    moved = (sum(lens) * ROW + T * H * (ROW + D_C)) * e + T * H * 4
    return {"bytes": moved, "flops": 2 * pairs * H * (ROW + D_C)}


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------
def _turn64(x, pos):
    x = x.double()
    i = torch.arange(D_R // 2, device=x.device, dtype=torch.float64)
    z = torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous())
    ang = pos.double()[:, None] * torch.pow(torch.tensor(THETA, dtype=torch.float64), -2 * i / D_R)
    turn = torch.polar(torch.ones_like(ang), ang)
    return torch.view_as_real(z * (turn if z.dim() == 2 else turn[:, None])).reshape(x.shape)


def _head64(q, k, v, first):
    """One head: row i of q sees the first + i + 1 first rows of k and v."""
    s = torch.tril(torch.ones(q.shape[0], k.shape[0], device=q.device, dtype=torch.bool), first)
    s = torch.where(s, (q @ k.T) / math.sqrt(D_QK), -math.inf)
    lse = torch.logsumexp(s, 1)
    return torch.exp(s - lse[:, None]) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    H, dev, at = s["H"], s["cu"].device, 0
    if case["op"] == "append":
        pool, k_rope = s["pool"].double(), torch.empty(s["T"], D_R, dtype=torch.float64, device=dev)
        q_rope = torch.empty(s["T"], H, D_R, dtype=torch.float64, device=dev)
        for b, n in enumerate(s["n"]):
            pos = torch.arange(s["lens_host"][b] - n, s["lens_host"][b], device=dev)
            one = slice(at, at + n)
            k_rope[one] = _turn64(s["k_r"][one], pos)
            q_rope[one] = _turn64(s["q"][one, :, D_N:], pos)
            page = s["table"][b].long()[pos // PAGE]
            pool[page, pos % PAGE, :D_C] = s["c_kv"][one].double()
            pool[page, pos % PAGE, D_C:] = k_rope[one]
            at += n
        return {"pool": pool, "k_rope": k_rope, "q_rope": q_rope}
    o = torch.empty(*s["o"].shape, dtype=torch.float64, device=dev)
    lse = torch.empty(s["T"], H, dtype=torch.float64, device=dev)
    for b, n in enumerate(s["n"]):
        one, first = slice(at, at + n), 0
        if case["op"] == "chunk":
            first = s["lens_host"][b] - n
            rows = s["pool"][s["table"][b, :-(-s["lens_host"][b] // PAGE)].long()]
            rows = rows.reshape(-1, ROW)[:s["lens_host"][b]].double()
        for h in range(H):
            if case["op"] == "chunk":
                q, k, v = s["q_cat"][one, h].double(), rows, rows[:, :D_C]
            else:
                hk = h * case["kv_heads"] // H
                q, v = s["q"][one, h].double(), s["v"][one, hk].double()
                k = torch.cat((s["k_nope"][one, hk], s["k_rope"][one]), 1).double()
            o[one, h], lse[one, h] = _head64(q, k, v, first)
        at += n
    return {"o": o, "lse": lse}
