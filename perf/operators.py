"""Measured cases of the operators around the sparse attention: the query/key
norms with the position rotation (and its backward), the quantised paged
cache (written and read back), the decode attention over that cache and the
top-k whose rows know their sequence's length.

`run` computes an operator in its plain form, from elementary torch
operations, or, where `own` is true, by the package's own call.
"""
from __future__ import annotations

import math

import torch

own = False

PAGE = 64            # tokens of a cache page (and of a selection block)
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases

def listed():
    heads = {"Hq": 32, "Hkv": 8, "d": 128}
    few = {"Hq": 28, "Hkv": 4, "d": 128}
    return [
        # one new token of 16 sequences, far into their contexts: latency counts
        dict(name="encode_step", op="encode", B=16, N=1, **heads, dtype="bf16", layout="half", rot=128, norm=True,
             far=131072, factor=8.0),
        # a whole 32K prompt in front of the prefill selector
        dict(name="encode_prompt", op="encode", B=1, N=32768, **heads, dtype="bf16", layout="half", rot=128,
             norm=True, far=32768, factor=8.0),
        # an odd length in fp32, part of the head rotated in neighbouring pairs: a small training step
        dict(name="encode_grad_f32", op="encode_grad", B=2, N=1021, **few, dtype="f32", layout="pairs", rot=64,
             norm=True, far=1021, factor=1.0),
        # the gated training workload's projection gradient
        dict(name="encode_grad", op="encode_grad", B=2, N=16384, **few, dtype="bf16", layout="half", rot=128,
             norm=True, far=16384, factor=1.0),
        # a decode step's new keys and values, sequences at their own offsets inside a page
        dict(name="append_step", op="append", B=16, T=1, Hkv=8, d=128, lo=1, hi=4095, blocks=64),
        # a padded batch of prompts written behind cached prefixes, pages that start and end inside the append
        dict(name="append_prompts", op="append", B=4, T=8191, Hkv=8, d=128, lo=37, hi=2100, blocks=161),
        # cached contexts read back in front of a prefill over them
        dict(name="read_context", op="read", B=4, T=16001, Hkv=8, d=128, lo=9000, hi=16384, blocks=256),
        # one sequence of an odd length, every block: the smallest decode
        dict(name="decode_one", op="decode", B=1, **heads, lo=4001, hi=4001, blocks=64, keep=0),
        # the decode workload: 96 kept blocks and the last of up to 2048, every sequence its own length
        dict(name="decode_kept", op="decode", B=16, **heads, lo=40000, hi=131072, blocks=2048, keep=97),
        # every block of long ragged sequences: the whole cache is read
        dict(name="decode_all", op="decode", B=16, **heads, lo=30000, hi=131072, blocks=2048, keep=0),
        # the selection of a small batch over short contexts
        dict(name="select_short", op="select", B=4, Hkv=4, blocks=100, lo=1, hi=6400, kb=16),
        # the selection of the decode workload, for many more sequences
        dict(name="select_long", op="select", B=256, Hkv=8, blocks=2048, lo=40000, hi=131072, kb=96),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["encode", "encode", "encode_grad", "append", "read", "decode", "decode", "select"])
    Hkv = rng.choice([1, 2, 4, 8])
    if op in ("encode", "encode_grad"):
        N = 1 if op == "encode" and rng.random() < 0.3 else _spread(rng, 2, 16000)
        d = rng.choice([64, 128])
        return dict(op=op, B=_spread(rng, 1, 64 if N < 300 else 2), N=N, Hq=Hkv * rng.choice([1, 2, 4, 7]), Hkv=Hkv,
                    d=d, dtype=rng.choice(["bf16", "bf16", "f32"]), layout=rng.choice(["half", "pairs"]),
                    rot=rng.choice([d // 4, d // 2, d]), norm=rng.random() < 0.8, far=_spread(rng, max(N, 64), 1000000),
                    factor=rng.choice([1.0, 4.0, 8.0]))
    if op == "select":
        blocks = _spread(rng, 2, 8192)
        return dict(op=op, B=_spread(rng, 1, 64), Hkv=Hkv, blocks=blocks, lo=_spread(rng, 1, 64 * blocks) // 2,
                    hi=64 * blocks - rng.randrange(64), kb=_spread(rng, 1, 256))
    if op == "decode":
        blocks = _spread(rng, 1, 1024)
        B = _spread(rng, 1, min(64, 131072 // (blocks * Hkv)))
        hi = PAGE * blocks - rng.randrange(PAGE)
        return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 4, 7, 8, 16]), Hkv=Hkv, d=128, lo=_spread(rng, 1, hi) - 1,
                    hi=hi, blocks=blocks, keep=rng.choice([0, _spread(rng, 1, 128)]))
    T = 1 if op == "append" and rng.random() < 0.4 else _spread(rng, 2, 8000)
    blocks = T // PAGE + _spread(rng, 2, 64)
    hi = PAGE * blocks - (T if op == "append" else 0)
    return dict(op=op, B=_spread(rng, 1, 64 if T < 300 else 8), T=T, Hkv=Hkv, d=rng.choice([64, 128]),
                lo=_spread(rng, 1, hi) - 1, hi=hi, blocks=blocks)


def _lengths(c):
    """The sequences' lengths, spread over [lo, hi]: a case's own, whatever the seed."""
    return [c["lo"] + int((c["hi"] - c["lo"]) * ((b * 0.6180339887 + 0.99 * (b > 0)) % 1.0)) for b in range(c["B"])]


def _new_lengths(c):
    """How many of the T appended tokens each sequence of the padded batch has."""
    return [c["T"] - (b * 7919) % (c["T"] // 4 + 1) for b in range(c["B"])]


# -------------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _keys_like(gen, *shape):
    """Rows as a model's keys and values have them: unlike sizes from row to row, a few large channels."""
    x = _randn(gen, *shape)
    x *= torch.exp(0.5 * _randn(gen, *shape[:-1], 1))
    x[..., ::29] *= 6.0
    return x


def _two_to(e):
    """2^(e - 127) of exponent bytes, exactly."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _quantised(x):
    """(codes e4m3, exponent bytes) of rows x [..., d] fp32."""
    m, e = torch.frexp(x.abs().amax(-1))
    byte = (e - 9 + (m > 0.875).int() + 127).clamp(10, 246)
    byte = torch.where(m > 0, byte, 10)
    codes = (x / _two_to(byte)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, byte.to(torch.uint8)


def _frequencies(c):
    """Angles per position of the rotated pairs, slowed down by parts for long contexts: fast pairs keep their
    frequency, slow ones are divided by the factor, between them a ramp. With them the factor on cos and sin."""
    half = c["rot"] // 2
    f = 500000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    if c["factor"] == 1.0:
        return f.to(DEV), 1.0
    turns = 8192 * f / (2 * math.pi)
    ramp = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
    return (f * ramp + f / c["factor"] * (1 - ramp)).to(DEV), 0.1 * math.log(c["factor"]) + 1.0


def _encode_state(c, gen):
    B, N, Hq, Hkv, d, dt = c["B"], c["N"], c["Hq"], c["Hkv"], c["d"], DTYPES[c["dtype"]]
    H = Hq + 2 * Hkv
    s = {"qkv": torch.stack([_keys_like(gen, N, H, d).to(dt) for _ in range(B)])}
    first = torch.randint(0, max(1, c["far"] - N + 1), (B, 1), generator=gen, device=DEV)
    s["positions"] = (first + torch.arange(N, device=DEV)).to(torch.int32)
    s["q_weight"] = (1 + 0.2 * _randn(gen, d)).to(dt) if c["norm"] else None
    s["k_weight"] = (1 + 0.2 * _randn(gen, d)).to(dt) if c["norm"] else None
    s["inv_freq"], s["rope_scale"] = _frequencies(c)
    s["eps"] = 1e-6
    if c["op"] == "encode_grad":
        s["dq"], s["dk"], s["dv"] = (0.1 * _randn(gen, B, h, N, d) for h in (Hq, Hkv, Hkv))
    if own:
        from top_block_sparse_bsa_b200 import BSA_ROPE_HALF, BSA_ROPE_PAIRS, pipeline
        s["step"] = pipeline.QkvStep(s["qkv"], Hq, Hkv, q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                                     inv_freq=s["inv_freq"], positions=s["positions"], rope_scale=s["rope_scale"],
                                     layout=BSA_ROPE_HALF if c["layout"] == "half" else BSA_ROPE_PAIRS)
    return s


def _table(c, gen, spare=3):
    """Pages of the sequences' blocks, in no order, and the number of pages."""
    pages = c["B"] * c["blocks"] + spare
    return torch.randperm(pages, generator=gen, device=DEV)[:c["B"] * c["blocks"]].view(c["B"], -1).int(), pages


def _cache(c, gen, fill):
    """A paged quantised cache; with `fill`, each sequence's tokens are there and what lies behind them is NaN."""
    table, pages = _table(c, gen)
    shape = (pages, c["Hkv"], PAGE, c["d"])
    s = {"table": table, "lens": torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)}
    for name in ("k", "v"):
        codes = torch.full(shape, 0x7F if fill else 0, dtype=torch.uint8, device=DEV)
        exps = torch.full(shape[:3], 255 if fill else 10, dtype=torch.uint8, device=DEV)
        for b, n in enumerate(_lengths(c) if fill else []):
            used = -(-n // PAGE)
            if not used:
                continue
            x = _keys_like(gen, used, c["Hkv"], PAGE, c["d"])
            q, e = _quantised(x.to(torch.bfloat16).float())
            q = q.view(torch.uint8)
            if n % PAGE:
                q[-1, :, n % PAGE:], e[-1, :, n % PAGE:] = 0x7F, 255
            at = table[b, :used].long()
            codes[at], exps[at] = q, e
        s[name + "_pool"], s[name + "_exp"] = codes.view(torch.float8_e4m3fn), exps
    return s


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    if c["op"] in ("encode", "encode_grad"):
        s = _encode_state(c, gen)
    elif c["op"] == "append":
        s = _cache(c, gen, False)
        for name in ("k_new", "v_new"):
            s[name] = _keys_like(gen, c["B"], c["Hkv"], c["T"], c["d"]).to(torch.bfloat16)
        s["new_lens"] = torch.tensor(_new_lengths(c), dtype=torch.int32, device=DEV)
        s["pooled"] = torch.zeros((c["B"], c["Hkv"], c["blocks"], c["d"]), device=DEV)
    elif c["op"] == "read":
        s = _cache(c, gen, True)
        for name in ("k_out", "v_out"):
            s[name] = torch.zeros((c["B"], c["Hkv"], c["T"], c["d"]), dtype=torch.bfloat16, device=DEV)
        # behind a prefix that the reader has already, where the sequence is long enough for one
        s["starts"] = torch.tensor([max(0, n - c["T"] - 5) for n in _lengths(c)], dtype=torch.int32, device=DEV)
    elif c["op"] == "decode":
        s = _cache(c, gen, True)
        s["q"] = (1.5 * _randn(gen, c["B"], c["Hq"], c["d"])).to(torch.bfloat16)
        s["idx"] = _kept_lists(c, gen) if c["keep"] else None
        s["scale"] = 1.0 / math.sqrt(c["d"])
        if own:
            from top_block_sparse_bsa_b200 import pipeline
            s["step"] = pipeline.QuantDecodeStep(s["q"], s["k_pool"], s["v_pool"], s["k_exp"], s["v_exp"], s["table"],
                                                 s["lens"], kb=c["keep"] - 1 if c["keep"] else None)
    else:
        n = c["B"] * c["Hkv"]
        s = {"scores": _randn(gen, n, c["blocks"]), "lens": torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)}
        s["scores"] += 3.0 * (_randn(gen, n, c["blocks"]) > 2.0)
        s["idx"] = torch.empty((n, c["kb"] + 1), dtype=torch.int32, device=DEV)
        s["count"] = torch.empty((n,), dtype=torch.int32, device=DEV)
    s["case"] = c
    return s


def _kept_lists(c, gen):
    """Kept blocks as a selector gives them: ascending, the sequence's last block among them, -1 behind."""
    nb = torch.tensor([-(-n // PAGE) for n in _lengths(c)], device=DEV)[:, None, None]
    rank = torch.rand((c["B"], c["Hkv"], c["blocks"]), generator=gen, device=DEV)
    j = torch.arange(c["blocks"], device=DEV)
    rank = torch.where(j < nb, rank, 2.0)
    rank = torch.where(j == nb - 1, -1.0, rank)
    keep = min(c["keep"], c["blocks"])
    value, at = rank.topk(keep, dim=-1, largest=False)
    at = torch.where(value < 1.5, at, c["blocks"]).sort(-1).values
    at = torch.where(at < c["blocks"], at, -1)
    return torch.nn.functional.pad(at, (0, c["keep"] - keep), value=-1).int().contiguous()


# --------------------------------------------------------------- plain forms

def _rotate(y, cos, sin, layout, rot):
    """The first `rot` channels of y turned by the angles: pair i is (i, i + rot/2) or (2i, 2i + 1)."""
    if layout == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., :rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _angles(s):
    t = s["positions"].double()[..., None] * s["inv_freq"]
    return (t.cos() * s["rope_scale"]).float()[:, :, None], (t.sin() * s["rope_scale"]).float()[:, :, None]


def _encode_plain(s):
    c, dt = s["case"], s["qkv"].dtype
    cos, sin = _angles(s)
    parts = s["qkv"].split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)
    out = []
    for x, w in zip(parts[:2], (s["q_weight"], s["k_weight"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        out.append(_rotate(y, cos, sin, c["layout"], c["rot"]).to(dt).transpose(1, 2).contiguous())
    return {"q": out[0], "k": out[1], "v": parts[2].transpose(1, 2).contiguous()}


def _encode_grad_plain(s):
    c, dt = s["case"], s["qkv"].dtype
    cos, sin = _angles(s)
    parts = s["qkv"].split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)
    dx, dw = [], []
    for x, w, dz in zip(parts[:2], (s["q_weight"], s["k_weight"]), (s["dq"], s["dk"])):
        dy = _rotate(dz.transpose(1, 2), cos, -sin, c["layout"], c["rot"])
        if w is not None:
            x = x.float()
            r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
            dw.append((dy * x * r).sum((0, 1, 2), dtype=torch.float64).float())
            dy = dy * w.float()
            dy = r * (dy - x * r.square() * (dy * x).mean(-1, keepdim=True))
        dx.append(dy.to(dt))
    return {"d_qkv": torch.cat(dx + [s["dv"].transpose(1, 2).to(dt)], 2), "dw": dw}


def _append_plain(s):
    c = s["case"]
    T = c["T"]
    t = torch.arange(T, device=DEV)
    pos = s["lens"].long()[:, None] + t
    here = t < s["new_lens"][:, None]
    page = s["table"].long().gather(1, (pos // PAGE).clamp(max=c["blocks"] - 1))[here]
    offset = (pos % PAGE)[here]
    for name in ("k", "v"):
        codes, exps = _quantised(s[name + "_new"].float())
        s[name + "_pool"].view(torch.uint8)[page, :, offset] = codes.view(torch.uint8).transpose(1, 2)[here]
        s[name + "_exp"][page, :, offset] = exps.transpose(1, 2)[here]
    # the blocks that this append completes get the mean of their keys
    j = torch.arange(c["blocks"], device=DEV)
    end = (j + 1) * PAGE
    whole = (end > s["lens"][:, None]) & (end <= (s["lens"] + s["new_lens"])[:, None])
    at = s["table"].long()[whole]
    keys = s["k_pool"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * _two_to(s["k_exp"][at])[..., None]
    s["pooled"].transpose(1, 2)[whole] = keys.mean(2)
    return {n: s[n] for n in ("k_pool", "v_pool", "k_exp", "v_exp", "pooled")}


def _read_plain(s):
    c = s["case"]
    t = torch.arange(c["T"], device=DEV)
    pos = s["starts"].long()[:, None] + t
    here = pos < s["lens"][:, None]
    page = s["table"].long().gather(1, (pos // PAGE).clamp(max=c["blocks"] - 1))[here]
    offset = (pos % PAGE)[here]
    for name in ("k", "v"):
        x = s[name + "_pool"].view(torch.uint8)[page, :, offset].view(torch.float8_e4m3fn).float()
        x = x * _two_to(s[name + "_exp"][page, :, offset])[..., None]
        s[name + "_out"].transpose(1, 2)[here] = x.to(torch.bfloat16)
    return {"k": s["k_out"], "v": s["v_out"]}


def _decode_plain(s):
    c = s["case"]
    B, Hkv, G, d = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["d"]
    if s["idx"] is None:
        blocks = torch.arange(c["blocks"], device=DEV).expand(B, Hkv, -1)
    else:
        blocks = s["idx"].long()
    page = s["table"].long()[:, None].expand(B, Hkv, -1).gather(2, blocks.clamp(min=0))
    head = torch.arange(Hkv, device=DEV)[None, :, None]
    pos = blocks[..., None] * PAGE + torch.arange(PAGE, device=DEV)
    seen = ((blocks >= 0)[..., None] & (pos < s["lens"][:, None, None, None])).flatten(2)   # [B,Hkv,n]
    def rows(name):
        x = s[name + "_pool"].view(torch.uint8)[page, head].view(torch.float8_e4m3fn).float()
        x = (x * _two_to(s[name + "_exp"][page, head])[..., None]).flatten(2, 3)
        return torch.where(seen[..., None], x, 0.0)
    logits = s["q"].view(B, Hkv, G, d).float() @ rows("k").transpose(2, 3) * s["scale"]
    logits = torch.where(seen[:, :, None], logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, p @ rows("v") / total, 0.0)
    return {"o": o.view(B, -1, d).to(torch.bfloat16), "lse": (top + total.log()).view(B, -1)}


def _select_plain(s):
    c = s["case"]
    n = ((s["lens"].long() + PAGE - 1) // PAGE).repeat_interleave(c["Hkv"])[:, None]
    j = torch.arange(c["blocks"], device=DEV)
    order = torch.argsort(torch.where(j < n - 1, s["scores"], -math.inf), dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order))
    kept = (rank < torch.clamp(n - 1, max=c["kb"])) | (j == n - 1)
    idx = torch.where(kept, j, c["blocks"]).sort(-1).values[:, :c["kb"] + 1]
    idx = torch.nn.functional.pad(idx, (0, c["kb"] + 1 - idx.shape[1]), value=c["blocks"])
    return {"idx": torch.where(idx < c["blocks"], idx, -1).int(), "count": kept.sum(-1, dtype=torch.int32)}


# ------------------------------------------------------------ one pass of it

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"encode": _encode_plain, "encode_grad": _encode_grad_plain, "append": _append_plain,
                "read": _read_plain, "decode": _decode_plain, "select": _select_plain}[op](state)
    return _run_own(op, state)


def _run_own(op, s):
    import top_block_sparse_bsa_b200 as bsa
    c = s["case"]
    if op == "encode":
        b = s["step"].run()
        return {n: b[n] for n in ("q", "k", "v")}
    if op == "encode_grad":
        b = s["step"].backward(s["dq"], s["dk"], s["dv"])
        return {"d_qkv": b["d_qkv"], "dw": [b["d_q_weight"], b["d_k_weight"]] if c["norm"] else []}
    if op == "decode":
        b = s["step"].attend(idx=s["idx"])
        return {"o": b["o"], "lse": b["lse"]}
    if op == "select":
        bsa.bsa_topk_select_lens(s["scores"], c["B"] * c["Hkv"], c["blocks"], s["lens"], c["Hkv"], PAGE, c["kb"],
                                 s["idx"], c["kb"] + 1, s["count"])
        return {"idx": s["idx"], "count": s["count"]}
    shape = bsa.make_shape(c["B"], c["Hkv"], c["Hkv"], c["T"], c["blocks"] * PAGE, c["d"], PAGE, torch.bfloat16)
    if op == "append":
        bsa.bsa_paged_append_quant(shape, s["k_new"], s["v_new"], s["lens"], s["table"], s["k_pool"], s["v_pool"],
                                   s["k_exp"], s["v_exp"], s["pooled"], new_lens=s["new_lens"])
        return {n: s[n] for n in ("k_pool", "v_pool", "k_exp", "v_exp", "pooled")}
    bsa.bsa_paged_read_quant(shape, s["k_pool"], s["v_pool"], s["k_exp"], s["v_exp"], s["table"], s["lens"],
                             s["k_out"], s["v_out"], starts=s["starts"])
    return {"k": s["k_out"], "v": s["v_out"]}


# ---------------------------------------------------------------------- work

def work(case):
    c = dict(case)
    if c["op"] in ("encode", "encode_grad"):
        size = 2 if c["dtype"] == "bf16" else 4
        tokens = c["B"] * c["N"]
        qk, v = tokens * (c["Hq"] + c["Hkv"]) * c["d"], tokens * c["Hkv"] * c["d"]
        if c["op"] == "encode":
            return {"bytes": 2 * (qk + v) * size + 4 * tokens, "flops": 8 * qk}
        # the forward's values are read again where the norm needs them; the gradients come in fp32
        return {"bytes": 4 * (qk + v) + (qk if c["norm"] else 0) * size + (qk + v) * size + 4 * tokens,
                "flops": 16 * qk}
    row = 2 * c.get("d", 0) + 2     # a token's codes and exponent bytes of one head's key and value
    if c["op"] == "append":
        new, lens = _new_lengths(c), _lengths(c)
        done = sum((a + b) // PAGE - a // PAGE for a, b in zip(lens, new))
        # new rows in bf16, their codes, and the completed blocks' means
        return {"bytes": c["Hkv"] * (sum(new) * (4 * c["d"] + row) + done * 4 * c["d"]),
                "flops": c["Hkv"] * sum(new) * 6 * c["d"]}
    if c["op"] == "read":
        n = sum(min(c["T"], n) for n in _lengths(c))
        return {"bytes": max(1, c["Hkv"] * n * (row + 4 * c["d"])), "flops": c["Hkv"] * n * 2 * c["d"]}
    if c["op"] == "decode":
        keys = sum(n if not c["keep"] or -(-n // PAGE) <= c["keep"] else (c["keep"] - 1) * PAGE + (n - 1) % PAGE + 1
                   for n in _lengths(c))
        return {"bytes": c["Hkv"] * keys * row + c["B"] * c["Hq"] * (4 * c["d"] + 4),
                "flops": c["Hq"] * keys * 4 * c["d"]}
    cols = sum(-(-n // PAGE) for n in _lengths(c))
    return {"bytes": 4 * c["Hkv"] * cols + 4 * c["B"] * c["Hkv"] * (c["kb"] + 2), "flops": c["Hkv"] * cols}


# ----------------------------------------------------------- exact, 64 bits

def _turned(y, turn, layout, rot):
    """Rotation as a product of complex numbers."""
    pairs = y[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2) if layout == "half" else \
        y[..., :rot].unflatten(-1, (rot // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = (z.transpose(-1, -2) if layout == "half" else z).flatten(-2)
    return torch.cat([z, y[..., rot:]], -1)


def _exact_encode(c, s):
    x = s["qkv"].double().requires_grad_(c["op"] == "encode_grad")
    w = [v.double().requires_grad_(c["op"] == "encode_grad") for v in (s["q_weight"], s["k_weight"]) if v is not None]
    angle = s["positions"].double()[:, :, None, None] * s["inv_freq"]
    turn = torch.polar(torch.full_like(angle, s["rope_scale"]), angle)
    ends = [c["Hq"], c["Hq"] + c["Hkv"]]
    out = []
    for n, (a, b) in enumerate(((0, ends[0]), (ends[0], ends[1]))):
        y = x[:, :, a:b]
        if w:
            y = y / (y.pow(2).sum(-1, keepdim=True) / c["d"] + s["eps"]).sqrt() * w[n]
        out.append(_turned(y, turn, c["layout"], c["rot"]).transpose(1, 2))
    out.append(x[:, :, ends[1]:].transpose(1, 2))
    if c["op"] == "encode":
        return dict(zip(("q", "k", "v"), out))
    torch.autograd.backward(out, [s[n].double() for n in ("dq", "dk", "dv")])
    return {"d_qkv": x.grad, "dw": [v.grad for v in w]}


def _power(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _to_e4m3(y):
    """y, |y| <= 448, rounded to three bits behind the leading one, halves to even; steps of 2^-9 at the least."""
    step = _power(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
    return torch.round(y / step) * step


def _exact_append(c, s):
    got = {"k_exp": None, "v_exp": None}
    for name in ("k", "v"):
        pool = torch.zeros(s[name + "_pool"].shape, dtype=torch.float64, device=DEV)
        size = torch.ones(pool.shape[:3], dtype=torch.float64, device=DEV)
        for b, (n0, n) in enumerate(zip(_lengths(c), _new_lengths(c))):
            x = s[name + "_new"][b, :, :n].double()
            m, e = torch.frexp(x.abs().amax(-1, keepdim=True) / 448)
            unit = _power(e - (m == 0.5).int())     # the least power of two that brings the row within 448
            pos = torch.arange(n0, n0 + n, device=DEV)
            page = s["table"][b].long()[pos // PAGE]
            pool[page, :, pos % PAGE] = _to_e4m3(x / unit).transpose(0, 1)
            size[page, :, pos % PAGE] = unit[..., 0].transpose(0, 1)
        got[name + "_pool"] = pool
        if name == "k":
            got["pooled"] = torch.zeros(s["pooled"].shape, dtype=torch.float64, device=DEV)
            for b, (n0, n) in enumerate(zip(_lengths(c), _new_lengths(c))):
                j = slice(n0 // PAGE, (n0 + n) // PAGE)
                at = s["table"][b].long()[j]
                # a page's part that lay there before holds zeros
                got["pooled"][b][:, j] = ((pool[at] * size[at][..., None]).sum(2) / PAGE).transpose(0, 1)
    return got


def _exact_rows(c, s, name, b):
    """Sequence b's tokens [Hkv, n, d]."""
    n = _lengths(c)[b]
    at = s["table"][b].long()[:-(-n // PAGE)]
    x = s[name + "_pool"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
    x = x * _power(s[name + "_exp"][at].long() - 127)[..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_read(c, s):
    got = {}
    for name in ("k", "v"):
        out = torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device=DEV)
        for b, first in enumerate(s["starts"].tolist()):
            x = _exact_rows(c, s, name, b)[:, first:first + c["T"]]
            out[b, :, :x.shape[1]] = x
        got[name] = out
    return got


def _exact_decode(c, s):
    o = torch.zeros((c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["d"]), dtype=torch.float64, device=DEV)
    lse = torch.full(o.shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lengths(c)):
        if not n:
            continue
        k, v = _exact_rows(c, s, "k", b), _exact_rows(c, s, "v", b)
        x = torch.einsum("gid,gnd->gin", s["q"][b].double().unflatten(0, (c["Hkv"], -1)), k) * s["scale"]
        if s["idx"] is not None:
            of = torch.arange(n, device=DEV) // PAGE
            kept = torch.stack([torch.isin(of, row) for row in s["idx"][b]])
            x = x.masked_fill(~kept[:, None], -math.inf)
        lse[b] = torch.logsumexp(x, -1)
        o[b] = torch.einsum("gin,gnd->gid", torch.softmax(x, -1), v)
    return {"o": o.flatten(1, 2), "lse": lse.flatten(1)}


def exact(case, seed):
    c = dict(case)
    if c["op"] == "select":
        return None       # whole numbers only
    s = prepare(c, seed)
    return {"encode": _exact_encode, "encode_grad": _exact_encode, "append": _exact_append, "read": _exact_read,
            "decode": _exact_decode}[c["op"]](c, s)
