"""Cases for the serving operators: the append to a paged key/value cache with the rotation
applied on the way, the attention of new tokens over that cache, and the processing of logits
before a draw (penalties, bias, grammar mask, temperature).

`run` computes a case in plain torch operations, or, with `own` set, through RLTModel.  Sizes are
those of the workloads in workloads/configs.py (heads, head widths, vocabularies, windows of up to
4096 positions) and generic serving batches with shared key/value heads.
"""
import math

import numpy as np
import torch

own = False

ROPE_BASE = 10000.0


# ------------------------------------------------------------------ the cases
def listed():
    a = dict(op="append", pad=0)
    t = dict(op="attend", pad=0)
    z = dict(op="logits")
    return [
        # one sequence, one new token: a single decode step of the 24+24 replay model's encoder
        dict(a, name="append_step_b1", dtype="bf16", src="f32", heads=16, kv_heads=16, hd=128, page=64, B=1,
             q_lo=1, q_hi=1, ctx_lo=2048, ctx_hi=2048, lens=1),
        # a serving batch in its decode phase with shared key/value heads, sources in bf16, small pages
        dict(a, name="append_step_b256_shared", dtype="bf16", src="bf16", heads=32, kv_heads=8, hd=128, page=16, B=256,
             q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=4095, lens=2),
        # the next turns of seven conversations of the 300M model, ragged, with rows of padding behind them
        dict(a, name="append_turns_b7", dtype="bf16", src="f32", heads=16, kv_heads=16, hd=64, page=64, B=7, q_lo=1,
             q_hi=900, ctx_lo=0, ctx_hi=2000, lens=3, pad=37),
        # prompts of the 48+48 model: 32 x 1024 tokens at once
        dict(a, name="append_prompt_32k", dtype="bf16", src="f32", heads=16, kv_heads=16, hd=128, page=128, B=32,
             q_lo=1024, q_hi=1024, ctx_lo=0, ctx_hi=0, lens=4),
        # the float32 model's cache
        dict(a, name="append_f32_b12", dtype="f32", src="f32", heads=4, kv_heads=4, hd=16, page=16, B=12, q_lo=1,
             q_hi=300, ctx_lo=0, ctx_hi=600, lens=5),
        # one sequence, one new token over a short context
        dict(t, name="attend_step_b1", dtype="bf16", heads=16, kv_heads=16, hd=64, page=64, B=1, q_lo=1, q_hi=1,
             ctx_lo=170, ctx_hi=170, lens=6),
        # a serving batch in its decode phase: 64 ragged contexts, shared key/value heads
        dict(t, name="attend_step_b64_shared", dtype="bf16", heads=32, kv_heads=8, hd=128, page=16, B=64, q_lo=1, q_hi=1,
             ctx_lo=500, ctx_hi=8000, lens=7),
        # the next turns of conversations of the 300M model beside single tokens of others
        dict(t, name="attend_turns_b9", dtype="bf16", heads=16, kv_heads=16, hd=64, page=64, B=9, q_lo=1, q_hi=700,
             ctx_lo=0, ctx_hi=3300, lens=8, pad=21),
        # a long document behind a long context, heads of the 48+48 model
        dict(t, name="attend_long_8k", dtype="bf16", heads=16, kv_heads=16, hd=128, page=128, B=1, q_lo=8192, q_hi=8192,
             ctx_lo=8192, ctx_hi=8192, lens=9),
        # the float32 model: chunks over its cache
        dict(t, name="attend_f32_b6", dtype="f32", heads=4, kv_heads=4, hd=16, page=16, B=6, q_lo=1, q_hi=200, ctx_lo=0,
             ctx_hi=900, lens=10),
        # one sequence of the smallest vocabulary
        dict(z, name="logits_b1", V=512, B=1, hist=100, lse=True, penalties=True, bias="none", mask=False, lens=11),
        # 512 sequences of the replay vocabulary under a grammar, with penalties over 1024 tokens of history
        dict(z, name="logits_b512", V=32768, B=512, hist=1024, lse=True, penalties=True, bias="shared", mask=True,
             lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "logits"])
    lens = rng.randrange(1 << 30)
    if op == "logits":
        V = 8 * _log_int(rng, 32, 6144)
        B = _log_int(rng, 1, min(512, max(1, 16_000_000 // V)))
        return dict(op=op, V=V, B=B, hist=_log_int(rng, 1, 4096), lse=rng.random() < 0.7, penalties=rng.random() < 0.8,
                    bias=rng.choice(["none", "shared", "row"]), mask=rng.random() < 0.6, lens=lens)
    dtype = "f32" if rng.random() < 0.15 else "bf16"
    if dtype == "f32":
        hd, kv, g = rng.choice([16, 32, 64]), rng.choice([1, 2, 4]), rng.choice([1, 1, 2, 3])
    else:
        hd, kv, g = rng.choice([16, 32, 64, 64, 128, 128]), rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 1, 2, 4, 7, 8])
        g = min(g, 32 // kv)
    case = dict(op=op, dtype=dtype, heads=kv * g, kv_heads=kv, hd=hd, page=rng.choice([16, 32, 64, 128, 256]),
                lens=lens, pad=rng.choice([0, 0, 1, 13]))
    if op == "append":
        case["src"] = "f32" if dtype == "f32" or rng.random() < 0.6 else "bf16"
    most_ctx = 2000 if dtype == "f32" else 16000
    B = _log_int(rng, 1, 128)
    kind = rng.choice(["step", "chunk", "chunk"])
    q_hi = 1 if kind == "step" else _log_int(rng, 2, 1500)
    ctx_hi = _log_int(rng, 1, most_ctx)
    if op == "append":
        while B > 1 and B * (q_hi + ctx_hi) * kv * hd > 150_000_000:
            B //= 2
    else:
        # scores of the padded batch, and the gathered keys
        while B > 1 and (B * kv * g * q_hi * (q_hi + ctx_hi) > 1_200_000_000 or B * kv * hd * (q_hi + ctx_hi) > 150_000_000
                         or B * kv * g * q_hi * hd * (ctx_hi + q_hi / 2) > 60_000_000_000):
            B //= 2
    return dict(case, B=B, q_lo=1, q_hi=q_hi, ctx_lo=0, ctx_hi=ctx_hi)


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """(new tokens, tokens in the cache behind the append) of every sequence, from the case alone."""
    r = np.random.default_rng([case["lens"], case["B"]])
    q = r.integers(case["q_lo"], case["q_hi"] + 1, case["B"])
    ctx = r.integers(case["ctx_lo"], case["ctx_hi"] + 1, case["B"])
    return q.astype(np.int64), (ctx + q).astype(np.int64)


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _model(case, max_pos):
    """The handle a user's program holds: its rotary table and vocabulary are the case's."""
    from cross_token_latent_b200 import RLTModel
    from workloads import ModelConfig

    hd = case.get("hd", 16)
    cfg = ModelConfig(V=case.get("V", 64), d=hd, n_heads=1, head_dim=hd, L_E=1, L_D=1, F=64, W=4, G=1,
                      dtype=case.get("dtype", "f32"), rope_base=ROPE_BASE)
    return RLTModel(cfg, max_pos=max_pos)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "logits":
        return _prepare_logits(case, seed, gen)
    q_len, kv_len = _lengths(case)
    B, P, hd, H, Hkv = case["B"], case["page"], case["hd"], case["heads"], case["kv_heads"]
    N, dt = int(q_len.sum()) + case["pad"], _type(case["dtype"])
    pages = -(-kv_len // P)
    # pages are handed out in no order, and some belong to nobody
    cols = int(pages.max())
    n_pages = int(pages.sum()) + 3
    r = np.random.default_rng(seed)
    table = np.zeros((B, cols), np.int32)
    free = r.permutation(n_pages)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = free[at:at + pages[b]]
        at += pages[b]
    s = dict(case=case, N=N, max_q=int(q_len.max()), max_kv=int(kv_len.max()),
             table=torch.from_numpy(table).cuda(),
             q_start=torch.from_numpy(np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)).cuda(),
             kv_len=torch.from_numpy(kv_len.astype(np.int32)).cuda())

    def normal(shape, dtype, scale=1.0):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        x.normal_(0.0, scale, generator=gen)
        return x

    s["pool"] = normal((n_pages, 2, Hkv, P, hd), dt)
    if case["op"] == "append":
        # queries, keys and values are column ranges of one projection's output, as the encoder has them
        qkv = normal((N, (H + 2 * Hkv) * hd), _type(case["src"]))
        s["q"] = qkv[:, :H * hd].unflatten(1, (H, hd))
        s["k"] = qkv[:, H * hd:(H + Hkv) * hd].unflatten(1, (Hkv, hd))
        s["v"] = qkv[:, (H + Hkv) * hd:].unflatten(1, (Hkv, hd))
        s["out"] = torch.zeros((N, H, hd), dtype=dt, device="cuda")
    else:
        # peaked and flat rows alike: scores of a standard deviation of 1.5 to 3
        s["q"] = normal((N, H, hd), dt, 2.0)
        s["out"] = torch.zeros((N, H, hd), dtype=dt, device="cuda")
    if own:
        s["model"] = _model(case, s["max_kv"])
        s["batch"] = s["model"].paged_batch(s["table"], s["q_start"], s["kv_len"], N, s["max_q"], s["max_kv"], P, Hkv)
    return s


def _prepare_logits(case, seed, gen):
    B, V, T = case["B"], case["V"], case["hist"]
    r = np.random.default_rng([case["lens"], B])
    s = dict(case=case)
    z = torch.empty((B, V), device="cuda").normal_(0.0, 3.0, generator=gen)
    s["lse"] = torch.logsumexp(z, 1) if case["lse"] else None
    s["x"] = z - s["lse"][:, None] if case["lse"] else z
    s["out"] = torch.empty_like(z)
    s["tau"] = torch.from_numpy(r.uniform(0.6, 1.2, B).astype(np.float32)).cuda()
    s["bias"] = s["mask"] = s["tokens"] = None
    if case["bias"] != "none":
        rows = B if case["bias"] == "row" else 1
        bias = torch.empty((rows, V), device="cuda").normal_(0.0, 1.0, generator=gen)
        s["bias"] = bias * (torch.rand((rows, V), device="cuda", generator=gen) < 0.05)
    if case["mask"]:
        s["mask"] = torch.randint(-2**31, 2**31, (B, -(-V // 32)), dtype=torch.int64, device="cuda",
                                  generator=gen).to(torch.int32)
    if case["penalties"]:
        # histories repeat themselves: ids are drawn from a skewed distribution
        u = torch.rand((B, T), device="cuda", generator=gen)
        s["tokens"] = (V * u ** 4).to(torch.int32).clamp_(max=V - 1)
        n = r.integers(0, T + 1, B)
        s["tok_len"] = torch.from_numpy(n.astype(np.int32)).cuda()
        s["gen_start"] = torch.from_numpy((n * r.random(B)).astype(np.int32)).cuda()
        for name, lo, hi in (("repetition", 0.8, 1.5), ("presence", -0.5, 1.0), ("frequency", 0.0, 0.5)):
            s[name] = torch.from_numpy(r.uniform(lo, hi, B).astype(np.float32)).cuda()
    if own:
        s["model"] = _model(case, 8)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if op == "append":
        return _own_append(s) if own else _plain_append(s)
    if op == "attend":
        return _own_attend(s) if own else _plain_attend(s)
    return _own_logits(s) if own else _plain_logits(s)


def _own_append(s):
    s["model"].paged_append(s["batch"], s["pool"], s["k"], s["v"], q=s["q"], q_out=s["out"])
    return s["out"], s["pool"]


def _own_attend(s):
    return s["model"].paged_attention(s["batch"], s["pool"], s["q"], out=s["out"])


def _own_logits(s):
    history = {} if s["tokens"] is None else {k: s[k] for k in ("tokens", "tok_len", "gen_start", "repetition", "presence",
                                                               "frequency")}
    return s["model"].process_logits(s["x"], lse=s["lse"], bias=s["bias"], mask=s["mask"], tau=s["tau"], out=s["out"],
                                     **history)


def _rows(s):
    """Of every packed row: its sequence, its position, and whether it belongs to a sequence at all."""
    n = torch.arange(s["N"], device="cuda")
    b = torch.searchsorted(s["q_start"], n, right=True) - 1
    valid = b < s["case"]["B"]
    b = b.clamp(max=s["case"]["B"] - 1)
    pos = s["kv_len"][b] - s["q_start"][b + 1] + n
    return b, pos, valid


def _plain_append(s):
    case = s["case"]
    hd, P, dt = case["hd"], case["page"], s["pool"].dtype
    b, pos, valid = _rows(s)
    # a row behind the last sequence repeats the first one, into the same slot
    row = torch.where(valid, torch.arange(s["N"], device="cuda"), 0)
    b, pos = b[row], pos[row]
    freq = ROPE_BASE ** (-torch.arange(0, hd, 2, dtype=torch.float64, device="cuda") / hd)
    angle = pos[:, None].double() * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotate(x):
        lo, hi = x[..., :hd // 2].float(), x[..., hd // 2:].float()
        return torch.cat([lo * cos - hi * sin, lo * sin + hi * cos], -1).to(dt)

    s["out"].copy_(torch.where(valid[:, None, None], rotate(s["q"][row]), s["out"]))
    page, slot = s["table"][b, pos // P].long(), pos % P
    s["pool"][page, 0, :, slot] = rotate(s["k"][row])
    s["pool"][page, 1, :, slot] = s["v"][row].float().to(dt)
    return s["out"], s["pool"]


def _plain_attend(s):
    case = s["case"]
    B, P, hd, H, Hkv = case["B"], case["page"], case["hd"], case["heads"], case["kv_heads"]
    Tq, Tk = s["max_q"], s["max_kv"]
    kv = s["pool"][s["table"].long()]                                   # [B, pages, 2, Hkv, P, hd]
    k, v = (kv[:, :, i].transpose(1, 2).flatten(2, 3)[:, :, :Tk].float() for i in (0, 1))
    b, pos, valid = _rows(s)
    n = torch.arange(s["N"], device="cuda")
    i = torch.where(valid, n - s["q_start"][b], Tq)                     # padding goes to a row of its own
    q = torch.zeros((B, Tq + 1, H, hd), device="cuda")
    q[b, i] = s["q"].float()
    q = q[:, :Tq].unflatten(2, (Hkv, H // Hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    scores = q @ k.transpose(2, 3) / math.sqrt(hd)                      # [B, Hkv, group * Tq, Tk]
    q_len = s["q_start"][1:] - s["q_start"][:-1]
    at = (s["kv_len"] - q_len)[:, None] + torch.arange(Tq, device="cuda")
    seen = torch.arange(Tk, device="cuda") <= at[:, :, None]            # [B, Tq, Tk]
    scores = scores.unflatten(2, (H // Hkv, Tq)).masked_fill_(~seen[:, None, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (H // Hkv, Tq)) / total.clamp(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)                          # [B, Tq, H, hd]
    rows = o[b, i.clamp(max=Tq - 1)].to(s["out"].dtype)
    s["out"].copy_(torch.where(valid[:, None, None], rows, s["out"]))
    return s["out"]


def _plain_logits(s):
    case = s["case"]
    B, V = case["B"], case["V"]
    z = s["x"] + s["lse"][:, None] if s["lse"] is not None else s["x"].clone()
    if s["tokens"] is not None:
        t = torch.arange(case["hist"], device="cuda")
        ids = s["tokens"].long()
        there = t < s["tok_len"][:, None]
        seen = torch.zeros((B, V), dtype=torch.int32, device="cuda").scatter_add_(1, ids, there.int())
        new = there & (t >= s["gen_start"][:, None])
        count = torch.zeros((B, V), dtype=torch.int32, device="cuda").scatter_add_(1, ids, new.int())
        rep = s["repetition"][:, None]
        z = torch.where(seen > 0, torch.where(z > 0, z / rep, z * rep), z)
        z = z - s["presence"][:, None] * (count > 0) - s["frequency"][:, None] * count
    if s["bias"] is not None:
        z = z + s["bias"]
    if s["mask"] is not None:
        bits = s["mask"][:, :, None] >> torch.arange(32, dtype=torch.int32, device="cuda") & 1
        z = z.masked_fill(bits.flatten(1)[:, :V] == 0, -math.inf)
    z = z / s["tau"][:, None]
    top = z.amax(1, keepdim=True).clamp(min=-1e30)
    s["out"].copy_(z - (top + (z - top).exp().sum(1, keepdim=True).log()))
    return s["out"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "logits":
        B, V = case["B"], case["V"]
        n = 2 * 4 * B * V + 4 * B
        n += 4 * B if case["lse"] else 0
        n += {"none": 0, "shared": 4 * V, "row": 4 * B * V}[case["bias"]]
        n += B * V // 8 if case["mask"] else 0
        if case["penalties"]:
            r = np.random.default_rng([case["lens"], B])
            r.uniform(0.6, 1.2, B)
            n += 4 * int(r.integers(0, case["hist"] + 1, B).sum()) + 20 * B
        return {"bytes": n, "flops": 6 * B * V}
    q_len, kv_len = _lengths(case)
    N, hd, H, Hkv = int(q_len.sum()), case["hd"], case["heads"], case["kv_heads"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        src = 2 if case["src"] == "bf16" else 4
        return {"bytes": N * (H + 2 * Hkv) * hd * (src + size), "flops": 3 * N * (H + Hkv) * hd}
    pairs = int((q_len * (kv_len - q_len) + q_len * (q_len + 1) // 2).sum())
    return {"bytes": size * hd * (2 * N * H + 2 * Hkv * int(kv_len.sum())), "flops": 4 * hd * H * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    if case["op"] == "logits":
        return _exact_logits(case, seed)
    s = prepare(case, seed)
    q_len, kv_len = _lengths(case)
    if case["op"] == "append":
        return _exact_append(case, s, q_len, kv_len)
    return _exact_attend(case, s, q_len, kv_len)


def _exact_append(case, s, q_len, kv_len):
    hd, P = case["hd"], case["page"]
    q_out, pool = s["out"].double(), s["pool"].double()
    f = torch.exp(torch.arange(hd // 2, dtype=torch.float64, device="cuda") * (-2.0 * math.log(ROPE_BASE) / hd))
    start = 0
    for b in range(case["B"]):
        rows = slice(start, start + int(q_len[b]))
        start = rows.stop
        pos = torch.arange(int(kv_len[b] - q_len[b]), int(kv_len[b]), device="cuda")
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None] * f)[:, None]

        def turned(x):
            y = torch.complex(x[rows, :, :hd // 2].double(), x[rows, :, hd // 2:].double()) * turn
            return torch.cat([y.real, y.imag], 2)

        q_out[rows] = turned(s["q"])
        page = s["table"][b, torch.div(pos, P, rounding_mode="floor")].long()
        pool[page, 0, :, pos % P] = turned(s["k"])
        pool[page, 1, :, pos % P] = s["v"][rows].double()
    return q_out, pool


def _exact_attend(case, s, q_len, kv_len):
    P, hd, Hkv = case["page"], case["hd"], case["kv_heads"]
    g = case["heads"] // Hkv
    if work(case)["flops"] > 1.5e12:
        return None
    out = s["out"].double()
    start = 0
    for b in range(case["B"]):
        nq, nk = int(q_len[b]), int(kv_len[b])
        pages = s["table"][b, :-(-nk // P)].long()
        ahead = torch.ones((nq, nk), dtype=torch.bool, device="cuda").triu(nk - nq + 1)
        for h in range(Hkv):
            k = s["pool"][pages, 0, h].reshape(-1, hd)[:nk].double()
            v = s["pool"][pages, 1, h].reshape(-1, hd)[:nk].double()
            for j in range(h * g, h * g + g):
                w = torch.einsum("qd,kd->qk", s["q"][start:start + nq, j].double(), k) * hd ** -0.5
                out[start:start + nq, j] = torch.softmax(w.masked_fill_(ahead, -math.inf), 1) @ v
        start += nq
    return out


def _exact_logits(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if s["lse"] is not None:
        x += s["lse"].double().unsqueeze(1)
    if s["tokens"] is not None:
        V = case["V"]
        tokens = s["tokens"].cpu().numpy()
        for b in range(case["B"]):
            n, new = int(s["tok_len"][b]), int(s["gen_start"][b])
            seen = torch.from_numpy(np.bincount(tokens[b, :n], minlength=V) > 0).cuda()
            count = torch.from_numpy(np.bincount(tokens[b, new:n], minlength=V)).cuda().double()
            rep = s["repetition"][b].double()
            x[b] = torch.where(seen, torch.where(x[b] > 0, x[b] / rep, x[b] * rep), x[b])
            x[b] -= s["presence"][b].double() * count.clamp(max=1) + s["frequency"][b].double() * count
    if s["bias"] is not None:
        x += s["bias"].double()
    if s["mask"] is not None:
        words = s["mask"].cpu().numpy().view(np.uint8).reshape(case["B"], -1)
        allowed = np.unpackbits(words, axis=1, bitorder="little")[:, :case["V"]]
        x[torch.from_numpy(allowed == 0).cuda()] = -math.inf
    return torch.log_softmax(x / s["tau"].double().unsqueeze(1), 1)
