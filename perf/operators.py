"""Cases of the serving operators: prompt attention, and the 4-bit cache's append, attention, eviction and read.

Each case is one pass through one operator.  `run` computes it in plain torch operations (float32, rounded once at the
end) or, where `own` is true, by the library's calls.  Both read the same state: packed rows, and a cache in the
library's 4-bit layout, which the plain forms unpack with shifts and masks.

The cache of one tensor, per (sequence, key/value head, row): d_h codes of 4 bits (code + 8) and one bfloat16 scale for
each group of 32 channels.  A row of K codes is d_h / 8 words of 8 nibbles; word t * (d_h / 32) + j holds channels
32 j + 8 t .. + 7, lowest nibble first.  A row of V codes is d_h / 4 halfwords of 4 nibbles; halfword g * (d_h / 32) + j
holds channels 32 j + 4 g .. + 3.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------
def listed():
    def prompt(name, lens, hist, H, H_kv, d, dtype, weight):
        return {"name": name, "op": "prompt", "lens": lens, "hist": hist, "H": H, "H_kv": H_kv, "d": d, "dtype": dtype,
                "weight": weight}

    return [
        # the float32 configuration's heads: a chat's first short turns, one of them a single token
        prompt("prompt short f32", "128,1,61", 0, 4, 4, 64, "f32", True),
        # a batch of prompts of different lengths, 16 heads of 64
        prompt("prompt ragged batch", "1024,17,640,333,1,900,512,1000,75,256,801,1023,128,400,64,711", 0, 16, 16, 64,
               "bf16", True),
        # one long document, grouped heads of 128, with the weights the eviction needs
        prompt("prompt long grouped", "8192", 0, 32, 8, 128, "bf16", True),
        # a batch's prompts go into the cache
        {"name": "append prompts", "op": "append", "B": 16, "n": 1024, "old": 0, "H_kv": 16, "d": 64, "cap": 2048,
         "dtype": "bf16"},
        # one generated token per sequence
        {"name": "append one token", "op": "append", "B": 16, "n": 1, "old": 1024, "H_kv": 16, "d": 64, "cap": 2048,
         "dtype": "bf16"},
        # the float32 configuration, one sequence: latency
        {"name": "attend one f32", "op": "attend", "B": 1, "n": 511, "H": 12, "H_kv": 12, "d": 64, "cap": 640,
         "dtype": "f32", "ragged": False},
        # a generating batch after prompts of about a thousand tokens
        {"name": "attend batch", "op": "attend", "B": 16, "n": 1152, "H": 16, "H_kv": 16, "d": 64, "cap": 1152,
         "dtype": "bf16", "ragged": True},
        # long contexts, grouped heads
        {"name": "attend long grouped", "op": "attend", "B": 32, "n": 16384, "H": 32, "H_kv": 8, "d": 128, "cap": 16384,
         "dtype": "bf16", "ragged": True},
        # the cache is halved
        {"name": "evict half", "op": "evict", "B": 16, "n": 1152, "keep": 576, "recent": 64, "H_kv": 16, "d": 64,
         "cap": 1152},
        # a long prompt's cache moves into a smaller one
        {"name": "evict long", "op": "evict", "B": 4, "n": 16384, "keep": 4096, "recent": 512, "H_kv": 8, "d": 128,
         "cap": 16384},
        # a short history is read back before a prompt goes on over it
        {"name": "read short", "op": "read", "B": 2, "n": 301, "H_kv": 8, "d": 128, "cap": 512, "dtype": "bf16"},
        # a batch's caches, whole
        {"name": "read batch", "op": "read", "B": 16, "n": 1024, "H_kv": 16, "d": 64, "cap": 1024, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "append", "attend", "attend", "evict", "read"))
    d = rng.choice((64, 128))
    H_kv = rng.choice((1, 2, 4, 8, 12, 16))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "prompt":
        G = rng.choice([g for g in (1, 2, 3, 4, 8) if g * H_kv <= 32])
        top = _log_int(rng, 8, 512 if dtype == "f32" else 6000)
        hist = rng.choice((0, 0, _log_int(rng, 1, 1500)))
        n_kv = top + hist
        most = max(1, min(16, int(2 ** 31 / (4 * H_kv * G * top * n_kv))))
        lens = [top] + [_log_int(rng, 1, top) for _ in range(rng.randint(1, most) - 1)]
        rng.shuffle(lens)
        return {"op": "prompt", "lens": ",".join(map(str, lens)), "hist": hist, "H": H_kv * G, "H_kv": H_kv, "d": d,
                "dtype": dtype, "weight": rng.random() < 0.7}
    if op == "append":
        n = rng.choice((1, _log_int(rng, 2, 2000)))
        old = rng.choice((0, rng.randint(1, 2000)))
        return {"op": "append", "B": rng.randint(1, 16), "n": n, "old": old, "H_kv": H_kv, "d": d,
                "cap": n + old + rng.randint(0, 50), "dtype": dtype}
    n = _log_int(rng, 8, 16000)
    B = rng.randint(1, max(1, min(32, int((8e6 if op == "attend" else 1e6) / (n * H_kv * d / 64)))))
    cap = n + rng.randint(0, 100)
    if op == "attend":
        G = rng.choice([g for g in (1, 2, 3, 4, 8, 16) if g * H_kv <= 64])
        return {"op": "attend", "B": B, "n": n, "H": H_kv * G, "H_kv": H_kv, "d": d, "cap": cap, "dtype": dtype,
                "ragged": rng.random() < 0.6}
    if op == "evict":
        keep = max(1, int(n * rng.uniform(0.1, 0.95)))
        return {"op": "evict", "B": B, "n": n, "keep": keep, "recent": int(keep * rng.uniform(0, 0.3)), "H_kv": H_kv,
                "d": d, "cap": cap}
    return {"op": "read", "B": B, "n": n, "H_kv": H_kv, "d": d, "cap": cap, "dtype": dtype}


# ---- state ---------------------------------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _keys(gen, *shape):
    """Keys have a few wide channels, as a projection's keys do."""
    x = _normal(gen, *shape)
    x[..., ::16] *= 3.0
    return x


def _ragged(case, gen):
    """The rows of each sequence: a half to all of n, the first one all of it."""
    B, n = case["B"], case["n"]
    if not case.get("ragged"):
        return torch.full((B,), n, dtype=torch.int32, device=DEV)
    u = torch.rand(B, generator=gen, device=DEV)
    ln = (n * (0.5 + 0.5 * u)).to(torch.int32).clamp(1, n)
    ln[0] = n
    return ln


def _quantise(x):
    """x [..., d] -> codes (float32, -7..7), scales (float32 holding bfloat16 values), by groups of 32 channels."""
    g = x.float().unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1) / torch.full((), 7.0, device=x.device)).to(torch.bfloat16).float()
    s = torch.where(s == 0, torch.ones_like(s), s)
    return torch.round(g / s[..., None]).clamp(-7, 7), s


def _pack(codes, run):
    """codes [..., groups, 32] -> bytes: runs of `run` channels, all groups' run t before any run t + 1."""
    u = (codes + 8).to(torch.uint8).unflatten(-1, (-1, run)).transpose(-3, -2).flatten(-3)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _unpack(b, d, run):
    """The codes (float32, -8..7) of packed rows, in channel order: [..., d / 32, 32]."""
    u = torch.stack((b & 15, b >> 4), -1).flatten(-2).unflatten(-1, (32 // run, d // 32, run))
    return u.transpose(-3, -2).flatten(-2).float() - 8


def _values(b, s, run):
    d = b.shape[-1] * 2
    return (_unpack(b, d, run) * s.float()[..., None]).flatten(-2)


def _new_cache(case, gen, n):
    """A cache that holds n rows of every sequence: packed codes, scales, weights and positions."""
    B, H, d, cap = case["B"], case["H_kv"], case["d"], case["cap"]
    c = {"k_codes": torch.full((B, H, cap, d // 2), 0x88, dtype=torch.uint8, device=DEV),
         "v_codes": torch.full((B, H, cap, d // 2), 0x88, dtype=torch.uint8, device=DEV),
         "k_scale": torch.ones((B, H, cap, d // 32), dtype=torch.bfloat16, device=DEV),
         "v_scale": torch.ones((B, H, cap, d // 32), dtype=torch.bfloat16, device=DEV),
         "weight": torch.zeros((B, H, cap), device=DEV),
         "pos": torch.zeros((B, H, cap), dtype=torch.int32, device=DEV)}
    if n:
        for b in range(B):   # one sequence at a time: the float32 rows of all of them are large
            for t, make, run in (("k", _keys, 8), ("v", _normal, 4)):
                q, s = _quantise(make(gen, H, n, d))
                c[t + "_codes"][b, :, :n] = _pack(q, run)
                c[t + "_scale"][b, :, :n] = s.to(torch.bfloat16)
        # accumulated weights fall off steeply; the positions of kept rows are spread over what was seen
        c["weight"][:, :, :n] = torch.exp(2.0 * _normal(gen, B, H, n))
        c["pos"][:, :, :n] = torch.arange(n, dtype=torch.int32, device=DEV)
    return c


def _handle(c):
    """The library's description of a cache."""
    from cascade_token_head_b200 import spatten as S
    return S.make_kv4_cache(c["k_codes"], c["k_scale"], c["v_codes"], c["v_scale"], c["weight"], c["pos"])


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, d = case["op"], case["d"]
    dt = DTYPES[case.get("dtype", "bf16")]
    s = {"case": case, "plan": None}
    if op == "prompt":
        lens = [int(x) for x in case["lens"].split(",")]
        kv = [x + case["hist"] for x in lens]
        s["lens"], s["kv"] = lens, kv
        s["q"] = (1.3 * _normal(gen, sum(lens), case["H"], d)).to(dt)
        s["k"] = _keys(gen, sum(kv), case["H_kv"], d).to(dt)
        s["v"] = _normal(gen, sum(kv), case["H_kv"], d).to(dt)
        s["cu_q"] = _i32([0] + torch.tensor(lens).cumsum(0).tolist())
        s["cu_kv"] = _i32([0] + torch.tensor(kv).cumsum(0).tolist())
        s["o"] = torch.empty_like(s["q"])
        s["w"] = torch.zeros((len(lens), case["H_kv"], max(kv)), device=DEV)
        return s
    B, H, n = case["B"], case["H_kv"], case["n"]
    if op == "append":
        s["cache"] = _new_cache(case, gen, case["old"])
        s["k"], s["v"] = _keys(gen, B * n, H, d).to(dt), _normal(gen, B * n, H, d).to(dt)
        s["cu"] = None if n == 1 else _i32([n * b for b in range(B + 1)])
        s["cu_read"] = _i32([n * b for b in range(B + 1)])
        s["len"] = _i32([case["old"]] * B)
        s["seen"] = _i32([case["old"] + 5 * b for b in range(B)])
        s["len_out"], s["seen_out"] = torch.zeros_like(s["len"]), torch.zeros_like(s["seen"])
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    elif op == "attend":
        s["cache"] = _new_cache(case, gen, n)
        s["len"] = _ragged(case, gen)
        s["q"] = (1.3 * _normal(gen, B, case["H"], d)).to(dt)
        s["o"] = torch.empty_like(s["q"])
    elif op == "evict":
        s["cache"] = _new_cache(case, gen, n)
        s["small"] = _new_cache(dict(case, cap=case["keep"]), gen, 0)
        s["len"] = _i32([n] * B)
        s["seen"] = _i32([n] * B)
        s["len_out"] = torch.zeros_like(s["len"])
        s["cu_read"] = _i32([case["keep"] * b for b in range(B + 1)])
        s["k_out"] = torch.empty((B * case["keep"], H, d), dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        s["cache"] = _new_cache(case, gen, n)
        s["cu_read"] = _i32([n * b for b in range(B + 1)])
        s["k_out"] = torch.empty((B * n, H, d), dtype=dt, device=DEV)
        s["v_out"] = torch.empty_like(s["k_out"])
    return s


# ---- the plain forms -------------------------------------------------------------------------------
def _softmax(x):
    """Rows of x and their exponentials' sums; a row of -inf only gives zeros."""
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = e.sum(-1, keepdim=True)
    return e / torch.where(l == 0, torch.ones_like(l), l)


def _plain_prompt(s):
    case = s["case"]
    H, Hk, d = case["H"], case["H_kv"], case["d"]
    G, nq, nk, B = H // Hk, max(s["lens"]), max(s["kv"]), len(s["lens"])
    lq, lk = (s["cu_q"][1:] - s["cu_q"][:-1]).long(), (s["cu_kv"][1:] - s["cu_kv"][:-1]).long()
    i, j = torch.arange(nq, device=DEV), torch.arange(nk, device=DEV)
    in_q, in_k = i < lq[:, None], j < lk[:, None]
    at_q = torch.where(in_q, s["cu_q"][:-1, None].long() + i, 0)
    at_k = torch.where(in_k, s["cu_kv"][:-1, None].long() + j, 0)
    q = s["q"].float()[at_q].view(B, nq, Hk, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * nq, d)
    k = s["k"].float()[at_k].transpose(1, 2)
    v = s["v"].float()[at_k].transpose(1, 2)
    x = (q @ k.transpose(-1, -2)).view(B, Hk, G, nq, nk).mul_(1 / math.sqrt(d))
    seen = in_q[:, :, None] & in_k[:, None, :] & (j <= i[:, None] + (lk - lq)[:, None, None])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    p = _softmax(x)
    del x
    o = (p.view(B, Hk, G * nq, nk) @ v).view(B, Hk, G, nq, d).permute(0, 3, 1, 2, 4).reshape(B, nq, H, d)
    out = {"o": o[in_q].to(s["q"].dtype)}
    if case["weight"]:
        s["w"] += p.sum((2, 3))
        out["weight"] = s["w"]
    return out


def _plain_append(s):
    c, case = s["cache"], s["case"]
    B, n, H, d, old = case["B"], case["n"], case["H_kv"], case["d"], case["old"]
    out = {}
    row = s["len"].long()[:, None] + torch.arange(n, device=DEV)
    b = torch.arange(B, device=DEV)[:, None]
    for t, run in (("k", 8), ("v", 4)):
        q, sc = _quantise(s[t].view(B, n, H, d))
        c[t + "_codes"][b, :, row] = _pack(q, run)
        c[t + "_scale"][b, :, row] = sc.to(torch.bfloat16)
        out[t] = _values(c[t + "_codes"][b, :, row], c[t + "_scale"][b, :, row], run).to(s[t].dtype).view(B * n, H, d)
    c["weight"][b, :, row] = 0.0
    pos = (s["seen"][:, None] + torch.arange(n, dtype=torch.int32, device=DEV))[:, :, None].expand(B, n, H)
    c["pos"][b, :, row] = pos
    return dict(out, weight=c["weight"], pos=c["pos"], len=s["len"] + n, seen=s["seen"] + n)


def _plain_attend(s):
    c, case = s["cache"], s["case"]
    B, H, Hk, d, n = case["B"], case["H"], case["H_kv"], case["d"], case["n"]
    q = s["q"].float().view(B, Hk, H // Hk, d)
    x = (q @ _values(c["k_codes"][:, :, :n], c["k_scale"][:, :, :n], 8).transpose(-1, -2)) / math.sqrt(d)
    x = x.masked_fill((torch.arange(n, device=DEV) >= s["len"][:, None])[:, None, None], -math.inf)
    p = _softmax(x)
    o = p @ _values(c["v_codes"][:, :, :n], c["v_scale"][:, :, :n], 4)
    c["weight"][:, :, :n] += p.sum(2)
    return {"o": o.view(B, H, d).to(s["q"].dtype), "weight": c["weight"]}


def _plain_evict(s):
    c, t, case = s["cache"], s["small"], s["case"]
    B, H, n, k = case["B"], case["H_kv"], case["n"], case["keep"]
    w = c["weight"][:, :, :n]
    safe = c["pos"][:, :, :n] >= (s["seen"] - case["recent"])[:, None, None]
    order = torch.where(safe, math.inf, w).sort(dim=-1, descending=True, stable=True)[1][..., :k]
    kept = torch.zeros((B, H, n), dtype=torch.bool, device=DEV).scatter_(-1, order, True)
    # the i-th hole below k takes the i-th kept row from k on
    hole = ~kept[..., :k]
    rank = hole.long().cumsum(-1) - 1
    behind = torch.where(kept[..., k:], torch.arange(k, n, device=DEV), n).sort(dim=-1)[0]
    behind = torch.nn.functional.pad(behind, (0, max(1, 2 * k - n)), value=n)
    src = torch.where(hole, behind.gather(-1, rank.clamp(min=0)), torch.arange(k, device=DEV))
    for key in ("k_codes", "k_scale", "v_codes", "v_scale"):
        t[key][:, :, :k] = c[key].gather(2, src[..., None].expand(-1, -1, -1, c[key].shape[-1]))
    for key in ("weight", "pos"):
        t[key][:, :, :k] = c[key].gather(2, src)
    values = [_values(t[x + "_codes"], t[x + "_scale"], run).to(torch.bfloat16).transpose(1, 2).reshape(B * k, H, -1)
              for x, run in (("k", 8), ("v", 4))]
    return {"k": values[0], "v": values[1], "weight": t["weight"], "pos": t["pos"], "len": s["len"].clamp(max=k)}


def _plain_read(s):
    c, case = s["cache"], s["case"]
    n, H, d = case["n"], case["H_kv"], case["d"]
    return {t: _values(c[t + "_codes"][:, :, :n], c[t + "_scale"][:, :, :n], run).to(s["k_out"].dtype)
            .transpose(1, 2).reshape(-1, H, d) for t, run in (("k", 8), ("v", 4))}


# ---- the library's calls ---------------------------------------------------------------------------
def _plan(s):
    """What a program sets up once for its buffers: argument structs and workspaces."""
    from cascade_token_head_b200 import spatten as S
    case, op = s["case"], s["case"]["op"]
    d, Hk = case["d"], case["H_kv"]
    if op == "prompt":
        a = S.make_prompt_args(s["q"], s["k"], s["v"], s["o"], s["cu_q"], s["cu_kv"],
                               weight=s["w"] if case["weight"] else None)
        nb = S.prompt_workspace_size(a)
        return a, torch.empty(max(nb, 256), dtype=torch.uint8, device=DEV), nb
    if op == "attend":
        a = S.make_kv4_attn_args(_handle(s["cache"]), s["q"], s["o"], s["len"], case["n"], update_weight=True)
        nb = S.kv4_attention_workspace_size(a)
        return a, torch.empty(max(nb, 256), dtype=torch.uint8, device=DEV), nb
    if op == "evict":
        src, dst = _handle(s["cache"]), _handle(s["small"])
        nb = S.kv4_evict_workspace_size(src, case["n"], case["keep"])
        return src, dst, torch.empty(max(nb, 256), dtype=torch.uint8, device=DEV), nb
    return (_handle(s["cache"]),)


def _own(s):
    from cascade_token_head_b200 import spatten as S
    case, op = s["case"], s["case"]["op"]
    if s["plan"] is None:
        s["plan"] = _plan(s)
    plan, HD = s["plan"], case["H_kv"] * case["d"]
    if op == "prompt":
        S.prompt_attention(*plan)
        return {"o": s["o"], "weight": s["w"]} if case["weight"] else {"o": s["o"]}
    if op == "append":
        total, c = case["B"] * case["n"], s["cache"]
        S.kv4_append(plan[0], s["k"], s["v"], HD, total, s["len"], s["len_out"], s["seen"], s["seen_out"], cu=s["cu"])
        S.kv4_read(plan[0], s["cu_read"], total, s["k_out"], s["v_out"], HD, row0=s["len"])
        return {"k": s["k_out"], "v": s["v_out"], "weight": c["weight"], "pos": c["pos"], "len": s["len_out"],
                "seen": s["seen_out"]}
    if op == "attend":
        S.kv4_attention(*plan)
        return {"o": s["o"], "weight": s["cache"]["weight"]}
    if op == "evict":
        src, dst, ws, nb = plan
        S.kv4_evict(src, dst, s["len"], s["len_out"], s["seen"], case["n"], case["keep"], case["recent"], ws, nb)
        S.kv4_read(dst, s["cu_read"], case["B"] * case["keep"], s["k_out"], s["v_out"], HD)
        return {"k": s["k_out"], "v": s["v_out"], "weight": s["small"]["weight"], "pos": s["small"]["pos"],
                "len": s["len_out"]}
    S.kv4_read(plan[0], s["cu_read"], case["B"] * case["n"], s["k_out"], s["v_out"], HD)
    return {"k": s["k_out"], "v": s["v_out"]}


_PLAIN = {"prompt": _plain_prompt, "append": _plain_append, "attend": _plain_attend, "evict": _plain_evict,
          "read": _plain_read}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without -------------------------------------------------------------------
def work(case):
    d, Hk = case["d"], case["H_kv"]
    es = 4 if case.get("dtype") == "f32" else 2
    row = 2 * (d // 2 + d // 16)        # codes and scales of one row's K and V
    if case["op"] == "prompt":
        lens = [int(x) for x in case["lens"].split(",")]
        pairs = sum(n * case["hist"] + n * (n + 1) / 2 for n in lens)
        kv = sum(lens) + len(lens) * case["hist"]
        w = case["weight"]
        return {"bytes": es * d * (2 * case["H"] * sum(lens) + 2 * Hk * kv) + (8 * Hk * kv if w else 0),
                "flops": 4 * d * case["H"] * pairs}
    rows = case["B"] * Hk * case["n"]
    if case["op"] == "append":          # rows in, codes, weights and positions written, values read back
        return {"bytes": rows * (2 * d * es + row + 8 + 2 * d * es), "flops": rows * 2 * d * 3}
    if case["op"] == "attend":
        mean = 0.75 if case["ragged"] else 1.0
        return {"bytes": mean * rows * (row + 8) + 2 * case["B"] * case["H"] * d * es,
                "flops": mean * rows * 4 * d * (case["H"] // Hk)}
    if case["op"] == "evict":           # weights and positions of all rows, kept rows moved and read back
        kept = case["B"] * Hk * min(case["keep"], case["n"])
        return {"bytes": rows * 8 + kept * (2 * (row + 8) + 4 * d), "flops": rows}
    return {"bytes": rows * (row + 2 * d * es), "flops": rows * 2 * d}


# ---- the definitions in 64 bits -------------------------------------------------------------------------
def _channels(codes, scale, run):
    """Values of packed rows in float64, channel by channel from the layout's definition."""
    d = codes.shape[-1] * 2
    c = torch.arange(d, device=codes.device)
    group, inside = c // 32, c % 32
    nibble = ((inside // run) * (d // 32) + group) * run + inside % run
    byte = codes[..., nibble // 2].to(torch.int64)
    return (((byte >> (4 * (nibble % 2))) & 15) - 8).double() * scale[..., group].double()


def _exact_prompt(s):
    case = s["case"]
    H, Hk, d = case["H"], case["H_kv"], case["d"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    w = torch.zeros(s["w"].shape, dtype=torch.float64, device=DEV)
    q0 = k0 = 0
    for b, (nq, nk) in enumerate(zip(s["lens"], s["kv"])):
        hidden = torch.ones((nq, nk), dtype=torch.bool, device=DEV).triu(nk - nq + 1)
        for h in range(H):
            k, v = (s[t][k0:k0 + nk, h * Hk // H].double() for t in "kv")
            x = (s["q"][q0:q0 + nq, h].double() @ k.T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
            p = torch.softmax(x, -1)
            o[q0:q0 + nq, h] = p @ v
            w[b, h * Hk // H, :nk] += p.sum(0)
        q0, k0 = q0 + nq, k0 + nk
    return {"o": o, "weight": w} if case["weight"] else {"o": o}


def _exact_append(s):
    case = s["case"]
    out = {"weight": s["cache"]["weight"].double(), "pos": None, "len": None, "seen": None}
    out["weight"][:, :, case["old"]:case["old"] + case["n"]] = 0
    for t in "kv":
        x = s[t].double().unflatten(-1, (-1, 32))
        scale = (x.abs().amax(-1, keepdim=True) / 7).float().to(torch.bfloat16).double()
        scale[scale == 0] = 1
        # the code is the rounded float32 quotient
        code = torch.clamp((x / scale).float().double().round(), -7, 7)
        out[t] = (code * scale).flatten(-2)
    return out


def _exact_attend(s):
    c, case = s["cache"], s["case"]
    B, H, Hk, d = case["B"], case["H"], case["H_kv"], case["d"]
    o = torch.zeros((B, H, d), dtype=torch.float64, device=DEV)
    w = c["weight"].double()
    for b, n in enumerate(s["len"].tolist()):
        for g in range(Hk):
            k = _channels(c["k_codes"][b, g, :n], c["k_scale"][b, g, :n], 8)
            v = _channels(c["v_codes"][b, g, :n], c["v_scale"][b, g, :n], 4)
            hs = slice(g * H // Hk, (g + 1) * H // Hk)
            p = torch.softmax(s["q"][b, hs].double() @ k.T / math.sqrt(d), -1)
            o[b, hs] = p @ v
            w[b, g, :n] += p.sum(0)
    return {"o": o, "weight": w}


def _exact_evict(s):
    c, case = s["cache"], s["case"]
    B, Hk, d, n, keep = case["B"], case["H_kv"], case["d"], case["n"], case["keep"]
    out = {t: torch.zeros((B, keep, Hk, d), dtype=torch.float64, device=DEV) for t in "kv"}
    w = torch.zeros((B, Hk, keep), dtype=torch.float64, device=DEV)
    weights, pos = c["weight"][:, :, :n].cpu(), c["pos"][:, :, :n].cpu()
    for b in range(B):
        for g in range(Hk):
            rows = [(p < n - case["recent"], 0.0 if p >= n - case["recent"] else -x, j)
                    for j, (x, p) in enumerate(zip(weights[b, g].tolist(), pos[b, g].tolist()))]
            kept = {j for _, _, j in sorted(rows)[:keep]}
            behind = iter(sorted(j for j in kept if j >= keep))
            src = torch.tensor([r if r in kept else next(behind) for r in range(keep)], device=DEV)
            w[b, g] = c["weight"][b, g, src].double()
            for t, run in (("k", 8), ("v", 4)):
                out[t][b, :, g] = _channels(c[t + "_codes"][b, g, src], c[t + "_scale"][b, g, src], run)
    return {"k": out["k"].flatten(0, 1), "v": out["v"].flatten(0, 1), "weight": w, "pos": None, "len": None}


def _exact_read(s):
    c, n = s["cache"], s["case"]["n"]
    return {t: _channels(c[t + "_codes"][:, :, :n], c[t + "_scale"][:, :, :n], run).transpose(1, 2).flatten(0, 1)
            for t, run in (("k", 8), ("v", 4))}


_EXACT = {"prompt": _exact_prompt, "append": _exact_append, "attend": _exact_attend, "evict": _exact_evict,
          "read": _exact_read}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
