"""Timed cases of four operators around the block-scaled cache, each beside its
plain form in elementary torch operations.

rotary    queries and keys rotated by their positions: pair i of a row, at the
          position p of the pair's axis (text: one axis; images and video: time,
          height, width), turns by the angle p * freq[i];
append    a prompt or a turn whose keys are rotated, rounded to bf16, and
          quantised with the values into the block-scaled cache (then read back
          as dense tensors), its queries rotated beside;
prefix    single-query attention of sequences that share a long prefix, held
          once, each followed by tokens of its own;
selected  single-query attention to the blocks of a long context that a cheap
          score selects, the newest blocks and the rows held exactly.

Definitions shared by all: 128 dims per head, query head j reads KV head
j / (Hq / Hkv); score = cap * tanh(s / cap) with s = q . k / sqrt(128) (s alone
where cap is 0), minus slope[j] * distance.  The cache: the first four positions
of a sequence and its open block are kept in bf16; a closed block of tokens has
one scale per KV head, amax / 127 (INT8) or amax / 448 (E4M3) in IEEE fp32, code
= x / scale (IEEE fp32 division) rounded half to even.

The cheap score of a closed block c for a query head: with q8 the INT8 codes of
the query row and s its scale, lo and hi the least and the largest INT8 code of
every channel of the block's keys (scale t = amax / 127, whatever codes the cache
holds), I = sum_d max(q8 lo, q8 hi), an upper bound of the dot product of the
codes; score = (I * s) * t, both products rounded to fp32.  A KV head takes the
largest of its query heads' scores; of equal ones the lower block comes first.
"""
import math
import random

import torch

own = False

D = 128
SINKS = 4
BASE = 10000.0


# --------------------------------------------------------------------- cases

def listed():
    return [
        # the queries and keys of one decoded token: the smallest call, all latency
        dict(name="rotary_one_token", op="rotary", batch=1, hq=8, hkv=8, n=1, rot=128, pairs="half", axes=1,
             first=511, fused=False),
        # prompts with an image (time, height, width), straight from a fused projection
        dict(name="rotary_image_prompts", op="rotary", batch=4, hq=32, hkv=8, n=4099, rot=128, pairs="half", axes=3,
             first=0, fused=True),
        # first tokens of many sequences after a prefix that they share
        dict(name="append_first_tokens", op="append", batch=64, hq=32, hkv=8, n=1, rot=128, pairs="half", axes=1,
             first=8192, fused=True, block=16, codes="int8"),
        # a short turn of many sequences, far into a long conversation
        dict(name="append_short_turns", op="append", batch=64, hq=8, hkv=8, n=41, rot=64, pairs="adjacent", axes=1,
             first=100000, fused=False, block=16, codes="int8"),
        # a batch of long prompts of a grouped-query model, from a fused projection
        dict(name="append_prompts_gqa", op="append", batch=8, hq=32, hkv=8, n=8192, rot=128, pairs="half", axes=1,
             first=0, fused=True, block=32, codes="int8"),
        # prompts with an image, as many KV heads as query heads, FP8 codes
        dict(name="append_image_prompts_e4m3", op="append", batch=4, hq=32, hkv=32, n=4001, rot=96, pairs="half",
             axes=3, first=0, fused=False, block=64, codes="e4m3"),
        # a few short sequences after a short prefix: latency
        dict(name="prefix_few_short", op="prefix", batch=4, hq=8, hkv=8, prefix=517, own=37, ragged=0, block=16,
             codes="int8", cap=0.0, bias=False),
        # a served batch after a long document
        dict(name="prefix_batch_long", op="prefix", batch=64, hq=32, hkv=8, prefix=32768, own=600, ragged=3, block=32,
             codes="int8", cap=0.0, bias=False),
        # five query heads on a KV head, FP8 codes, both transforms, odd sizes
        dict(name="prefix_gqa5_e4m3_cap_bias", op="prefix", batch=24, hq=40, hkv=8, prefix=16001, own=1100, ragged=7,
             block=64, codes="e4m3", cap=30.0, bias=True),
        # one sequence of ordinary length: latency
        dict(name="selected_one_seq", op="selected", batch=1, hq=32, hkv=8, ctx=8197, ragged=0, block=16, codes="int8",
             top=60, recent=4, cap=0.0, bias=False),
        # a served batch of long contexts
        dict(name="selected_batch_long", op="selected", batch=16, hq=32, hkv=8, ctx=65536, ragged=5, block=32,
             codes="int8", top=120, recent=8, cap=0.0, bias=False),
        # large blocks, FP8 codes, both transforms, five query heads on a KV head
        dict(name="selected_e4m3_cap_bias", op="selected", batch=8, hq=40, hkv=8, ctx=30001, ragged=9, block=64,
             codes="e4m3", top=62, recent=2, cap=50.0, bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "prefix", "selected"])
    hkv = rng.choice([1, 2, 4, 8, 16, 32])
    hq = hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8) if g * hkv <= 64])
    block, codes = rng.choice([16, 32, 64, 128]), rng.choice(["int8", "e4m3"])
    cap, bias = rng.choice([0.0, round(rng.uniform(4.0, 60.0), 2)]), rng.random() < 0.5
    if op in ("rotary", "append"):
        most = (1 << (21 if op == "append" else 19)) // (hq + 2 * hkv)
        n = _log_int(rng, 1, min(16384, most))
        batch = _log_int(rng, 1, max(1, min(64, most // n)))
        case = dict(op=op, batch=batch, hq=hq, hkv=hkv, n=n, rot=rng.choice([16, 32, 64, 96, 128]),
                    pairs=rng.choice(["half", "adjacent"]), axes=rng.choice([1, 3]), first=_log_int(rng, 1, 1000000) - 1,
                    fused=rng.random() < 0.5)
        return case if op == "rotary" else case | dict(block=block, codes=codes)
    if op == "prefix":
        prefix = _log_int(rng, 1, min(65536, (1 << 19) // hkv))
        batch = _log_int(rng, 1, max(1, min(64, (1 << 26) // (prefix * hq))))
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, prefix=prefix,
                    own=_log_int(rng, 1, max(1, min(8192, (1 << 18) // (batch * hkv)))),
                    ragged=rng.choice([0, rng.randrange(1, 1000)]), block=block, codes=codes, cap=cap, bias=bias)
    ctx = _log_int(rng, 1, min(131072, (1 << 21) // hkv))
    batch = _log_int(rng, 1, max(1, min(64, (1 << 21) // (ctx * hkv))))
    return dict(op=op, batch=batch, hq=hq, hkv=hkv, ctx=ctx, ragged=rng.choice([0, rng.randrange(1, 1000)]),
                block=block, codes=codes, top=_log_int(rng, 1, 4096 // block), recent=rng.randrange(0, 9), cap=cap,
                bias=bias)


def _lengths(case, most):
    """Tokens held per sequence: all `most`, or spread over [most / 8, most]."""
    if not case["ragged"]:
        return [most] * case["batch"]
    r = random.Random(case["ragged"])
    return [r.randint(max(1, most // 8), most) for _ in range(case["batch"])]


def _closed(tokens, block):
    return max(tokens - SINKS, 0) // block


def work(case):
    if case["op"] in ("rotary", "append"):
        rows = case["batch"] * case["n"]
        at = 4 * rows * case["axes"]
        turned = 3 * rows * (case["hq"] + case["hkv"]) * case["rot"]
        if case["op"] == "rotary":
            return {"bytes": 2 * 2 * D * rows * (case["hq"] + case["hkv"]) + at, "flops": turned}
        # queries in and out; keys and values in, codes out, codes in, dense rows out
        return {"bytes": D * rows * (4 * case["hq"] + 2 * case["hkv"] * (2 + 1 + 1 + 2)) + at,
                "flops": turned + 4 * D * rows * case["hkv"]}
    io = 2 * case["batch"] * case["hq"] * D * 2
    group, per = case["hq"] // case["hkv"], 2 * D + 8 / case["block"]
    if case["op"] == "prefix":
        tokens = sum(_lengths(case, case["own"]))
        seen = tokens + case["batch"] * case["prefix"]
        return {"bytes": (tokens + case["prefix"]) * case["hkv"] * per + io,
                "flops": 4 * seen * case["hkv"] * group * D}
    tokens = bounds = 0
    for n in _lengths(case, case["ctx"]):
        closed = _closed(n, case["block"])
        used = min(closed, case["top"] + case["recent"])
        tokens += n - (closed - used) * case["block"]
        bounds += closed if used < closed else 0
    return {"bytes": tokens * case["hkv"] * per + bounds * case["hkv"] * (2 * D + 4) + io,
            "flops": (4 * tokens + 2 * bounds) * case["hkv"] * group * D}


# -------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _keys(g, *shape):
    """Keys with four outlier channels, as trained models have them."""
    k = _randn(g, *shape)
    k[..., torch.randperm(D, generator=g, device="cuda")[:4]] *= 6.0
    return k.to(torch.bfloat16)


def _slopes(case):
    """The geometric slopes of the distance bias."""
    if not case["bias"]:
        return None
    return torch.tensor([2.0 ** (-8.0 * (j + 1) / case["hq"]) for j in range(case["hq"])], device="cuda")


def _axis_of_pairs(case):
    """The axis of every pair: one, or a quarter of the pairs for time and the
    rest for height and width."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return [0] * half
    return [0 if i < half // 4 else 1 + (i >= half // 4 + (half - half // 4) // 2) for i in range(half)]


def _freqs(case):
    """fp32 angles per position of every pair."""
    half = case["rot"] // 2
    return torch.tensor([BASE ** (-i / half) for i in range(half)], dtype=torch.float32)


def _positions(case):
    """int32 [axes, batch, n].  One axis: text from `first` on.  Three: an eighth
    of text, then an image whose rows and columns count on from its end."""
    at = torch.arange(case["n"], device="cuda", dtype=torch.int32)
    if case["axes"] == 3:
        text = case["n"] // 8
        wide = max(1, math.isqrt(case["n"] - text))
        patch = (at - text).clamp(min=0)
        image = torch.stack([torch.full_like(at, text), text + patch // wide, text + patch % wide])
        at = torch.where(at < text, at, image)
    else:
        at = at[None]
    return (at + case["first"])[:, None].expand(-1, case["batch"], -1).contiguous()


def _draw_rows(case, seed):
    """q, k, v (bf16, [batch, heads, n, 128]): one block each, or views of one
    projection's output [batch, n, heads, 128]."""
    g = _generator(seed)
    b, n, hq, hkv = case["batch"], case["n"], case["hq"], case["hkv"]
    q = _randn(g, b, n, hq, D).to(torch.bfloat16)
    k = _keys(g, b, n, hkv, D)
    v = _randn(g, b, n, hkv, D).to(torch.bfloat16)
    if case["fused"]:
        return [x.transpose(1, 2) for x in torch.cat([q, k, v], dim=2).split([hq, hkv, hkv], dim=2)]
    return [x.transpose(1, 2).contiguous() for x in (q, k, v)]


def _draw_held(case, seed):
    """q [batch, hq, 128], and (k, v, lengths) of the sequences in the cache: the
    prefix first, where there is one."""
    g = _generator(seed)
    q = _randn(g, case["batch"], case["hq"], D).to(torch.bfloat16)
    parts = [(case["batch"], case["own"] if case["op"] == "prefix" else case["ctx"])]
    if case["op"] == "prefix":
        parts.insert(0, (1, case["prefix"]))
    kv = []
    for count, n in parts:
        k = _keys(g, count, case["hkv"], n, D)
        v = _randn(g, count, case["hkv"], n, D).to(torch.bfloat16)
        kv.append((k, v, [n] if len(kv) + 1 < len(parts) else _lengths(case, n)))
    return q, kv


QMAX = {"int8": 127.0, "e4m3": 448.0}


def _codes(x, amax, codes):
    """(codes, scale) of fp32 values x whose largest magnitude is amax."""
    scale = amax / torch.full_like(amax, QMAX[codes])
    y = torch.where(scale > 0, x / scale, torch.zeros_like(x))
    if codes == "e4m3":
        return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale
    return y.round().clamp(-127.0, 127.0).to(torch.int8), scale


def _plain_cache(case, k, v, lengths, bounds):
    """The plain form's cache of sequences: codes [seqs, hkv, blocks, block, 128]
    and scales of all blocks, the exact rows [seqs, hkv, 4 + block, 128] (bf16)
    with their positions (-1: none), with `bounds` the least and largest INT8
    code of every channel of a block's keys and their scale."""
    block, n = case["block"], k.shape[2]
    blocks = -(-max(n - SINKS, 0) // block)
    held = dict(lengths=torch.tensor(lengths, device="cuda"))
    at = torch.arange(SINKS + block, device="cuda")
    closed = (held["lengths"] - SINKS).clamp(min=0)[:, None] // block * block
    at = torch.where(at < SINKS, at, at + closed)
    held["exact_at"] = torch.where(at < held["lengths"][:, None], at, -1)
    rows = held["exact_at"].clamp(min=0)[:, None, :, None].expand(-1, case["hkv"], -1, D)
    for name, x in (("k", k), ("v", v)):
        held[name + "_exact"] = x.gather(2, rows)
        body = torch.nn.functional.pad(x[:, :, SINKS:].float(), (0, 0, 0, blocks * block - max(n - SINKS, 0)))
        body = body.reshape(x.shape[0], case["hkv"], blocks, block, D)
        amax = body.abs().amax((-1, -2), keepdim=True)
        held[name + "_codes"], held[name + "_scale"] = _codes(body, amax, case["codes"])
        if bounds and name == "k":
            eights, scale = _codes(body, amax, "int8")
            held |= dict(lo=eights.amin(3), hi=eights.amax(3), bound_scale=scale[..., 0, 0])
    return held


def prepare(case, seed):
    state = dict(case=case)
    if case["op"] in ("rotary", "append"):
        q, k, v = _draw_rows(case, seed)
        freqs = _freqs(case)
        state |= dict(q=q, k=k, v=v, positions=_positions(case))
        if own:
            from compressed_kv_cache_kvc_gb300 import BlockScaledCache, Rotary
            state["rotary"] = Rotary(case["rot"], freqs=freqs.tolist(), axes=_axis_of_pairs(case),
                                     adjacent=case["pairs"] == "adjacent")
            if case["op"] == "append":
                per_seq = case["n"] // case["block"] + 1
                state["cache"] = BlockScaledCache(case["hq"], case["hkv"], case["batch"] * per_seq, case["batch"],
                                                  per_seq, block_tokens=case["block"], codes=case["codes"])
        else:
            state |= dict(freqs=freqs.cuda(), axis=torch.tensor(_axis_of_pairs(case), device="cuda"))
        return state
    q, kv = _draw_held(case, seed)
    state |= dict(q=q, slopes=_slopes(case))
    if not own:
        state["held"] = [_plain_cache(case, *x, case["op"] == "selected") for x in kv]
        return state
    from compressed_kv_cache_kvc_gb300 import BlockScaledCache
    counts = [_closed(n, case["block"]) for _, _, lengths in kv for n in lengths]
    cache = BlockScaledCache(case["hq"], case["hkv"], max(1, sum(counts)), len(counts), max(1, max(counts)),
                             block_tokens=case["block"], codes=case["codes"], key_bounds=case["op"] == "selected")
    seq = 0
    for k, v, lengths in kv:
        for b, n in enumerate(lengths):
            cache.append(k[b:b + 1, :, :n].contiguous(), v[b:b + 1, :, :n].contiguous(), seq_begin=seq)
            seq += 1
    state["cache"] = cache
    return state


# --------------------------------------------------------------- plain forms

def _plain_turn(state, x, cos, sin):
    """Rows x [batch, heads, n, 128] turned (cos, sin [batch, 1, n, rot / 2])."""
    rot = state["case"]["rot"]
    x = x.float()
    y = x.clone()
    if state["case"]["pairs"] == "adjacent":
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y.to(torch.bfloat16)


def _plain_rotary(state):
    angle = state["positions"][state["axis"]].permute(1, 2, 0).double() * state["freqs"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return _plain_turn(state, state["q"], cos, sin), _plain_turn(state, state["k"], cos, sin)


def _plain_append(state):
    case = state["case"]
    q, k = _plain_rotary(state)
    n, block = case["n"], case["block"]
    blocks = _closed(n, block)

    def read(t):
        x = t[:, :, SINKS:SINKS + blocks * block].float().reshape(case["batch"], case["hkv"], blocks, block, D)
        if blocks:
            c, scale = _codes(x, x.abs().amax((-1, -2), keepdim=True), case["codes"])
            x = c.float() * scale
        x = x.reshape(case["batch"], case["hkv"], blocks * block, D).to(torch.bfloat16)
        return torch.cat([t[:, :, :SINKS], x, t[:, :, SINKS + blocks * block:]], dim=2)

    return q, read(k), read(state["v"])


def _transform(s, case, slopes, distance):
    """Scores s (fp32 [batch, hkv, group, keys]), capped and biased."""
    if case["cap"]:
        s = torch.tanh(s / case["cap"]) * case["cap"]
    if slopes is not None:
        s = s - slopes.view(case["hkv"], -1, 1) * distance
    return s


def _plain_select(state, held):
    """int64 [batch, hkv, most] blocks, ascending, -1 behind the last."""
    case = state["case"]
    closed = (held["lengths"] - SINKS).clamp(min=0) // case["block"]
    q = state["q"].float().view(case["batch"], case["hkv"], -1, D)
    codes, scale = _codes(q, q.abs().amax(-1, keepdim=True), "int8")
    codes = codes.float()
    dots = codes.clamp(min=0) @ held["hi"].float().transpose(-1, -2)
    dots = dots + codes.clamp(max=0) @ held["lo"].float().transpose(-1, -2)
    score = ((dots * scale) * held["bound_scale"][:, :, None]).amax(2)
    blocks, most = score.shape[-1], case["top"] + case["recent"]
    at = torch.arange(blocks, device="cuda")
    end = closed.view(-1, 1, 1)
    score = torch.where(at >= end - case["recent"], math.inf, score)
    score = torch.where(at < end, score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :most]
    order = torch.sort(torch.where(order < end, order, blocks), dim=-1).values
    order = torch.nn.functional.pad(order, (0, most - order.shape[-1]), value=blocks)
    return torch.where(order < end, order, -1)


def _plain_selected(state):
    case, held = state["case"], state["held"][0]
    chosen = _plain_select(state, held)
    b, hkv, most = chosen.shape
    scale = 1.0 / math.sqrt(D)
    rows = []
    for name in ("k", "v"):
        exact = held[name + "_exact"].float()
        if held[name + "_codes"].shape[2]:
            at = (torch.arange(b, device="cuda")[:, None, None], torch.arange(hkv, device="cuda")[None, :, None],
                  chosen.clamp(min=0))
            body = held[name + "_codes"][at].float() * held[name + "_scale"][at]
            exact = torch.cat([body.reshape(b, hkv, most * case["block"], D), exact], dim=2)
        rows.append(exact)
    at = held["exact_at"][:, None].expand(-1, hkv, -1)
    if rows[0].shape[2] > at.shape[2]:
        body = SINKS + chosen[..., None] * case["block"] + torch.arange(case["block"], device="cuda")
        at = torch.cat([torch.where(chosen[..., None] >= 0, body, -1).flatten(2), at], dim=2)
    q = state["q"].float().view(b, hkv, -1, D)
    s = (q @ rows[0].transpose(-1, -2)) * scale
    distance = (held["lengths"].view(-1, 1, 1) - 1 - at).float()
    s = _transform(s, case, state["slopes"], distance[:, :, None])
    s = s.masked_fill(at[:, :, None] < 0, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    out = (p / p.sum(-1, keepdim=True)) @ rows[1]
    return out.reshape(b, case["hq"], D).to(torch.bfloat16), chosen.to(torch.int32)


def _dense(case, held, name):
    """fp32 [seqs, hkv, tokens, 128]: every closed block's rows, then the exact ones."""
    body = held[name + "_codes"].float() * held[name + "_scale"]
    return torch.cat([body.flatten(2, 3), held[name + "_exact"].float()], dim=2)


def _dense_at(case, held):
    """Positions of _dense's rows [seqs, tokens], -1 where there is none."""
    blocks = held["k_codes"].shape[2]
    at = SINKS + torch.arange(blocks * case["block"], device="cuda")
    closed = (held["lengths"] - SINKS).clamp(min=0)[:, None] // case["block"] * case["block"]
    return torch.cat([torch.where(at < SINKS + closed, at, -1), held["exact_at"]], dim=1)


def _plain_prefix(state):
    """The softmax over the prefix, computed for all queries at once, joined with
    the one over each sequence's own tokens."""
    case = state["case"]
    b, hkv = case["batch"], case["hkv"]
    q = state["q"].float().view(b, hkv, -1, D) * (1.0 / math.sqrt(D))
    shared, mine = state["held"]
    newest = case["prefix"] + mine["lengths"] - 1
    at = _dense_at(case, shared)[0]
    s = (q.permute(1, 0, 2, 3).flatten(1, 2) @ _dense(case, shared, "k")[0].transpose(-1, -2))
    s = s.view(hkv, b, -1, at.shape[0]).permute(1, 0, 2, 3)
    s = _transform(s, case, state["slopes"], (newest[:, None] - at).float()[:, None, None])
    s = s.masked_fill(at < 0, -math.inf)
    at = _dense_at(case, mine)
    t = q @ _dense(case, mine, "k").transpose(-1, -2)
    distance = (newest[:, None] - case["prefix"] - at).float()
    t = _transform(t, case, state["slopes"], distance[:, None, None])
    t = t.masked_fill((at < 0)[:, None, None], -math.inf)
    top = torch.maximum(s.amax(-1, keepdim=True), t.amax(-1, keepdim=True))
    s, t = torch.exp(s - top), torch.exp(t - top)
    total = s.sum(-1, keepdim=True) + t.sum(-1, keepdim=True)
    out = s.permute(1, 0, 2, 3).flatten(1, 2) @ _dense(case, shared, "v")[0]
    out = out.view(hkv, b, -1, D).permute(1, 0, 2, 3) + t @ _dense(case, mine, "v")
    return (out / total).reshape(b, case["hq"], D).to(torch.bfloat16)


# ----------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if not own:
        return {"rotary": _plain_rotary, "append": _plain_append, "prefix": _plain_prefix,
                "selected": _plain_selected}[case["op"]](state)
    if case["op"] == "rotary":
        return state["rotary"].rotate(state["q"], state["k"], positions=state["positions"])
    cache = state["cache"]
    if case["op"] == "append":
        cache.release(0, case["batch"])
        q = cache.append_rotary(state["q"], state["k"], state["v"], state["rotary"], positions=state["positions"])
        return q, *cache.read(0, case["batch"], 0, case["n"])
    if case["op"] == "prefix":
        return cache.prefix_attention(state["q"], prefix=0, seq_begin=1, softcap=case["cap"], slopes=state["slopes"])
    return cache.selected_attention(state["q"], case["top"], recent_blocks=case["recent"], softcap=case["cap"],
                                    slopes=state["slopes"], return_blocks=True)


# -------------------------------------------------------------- in 64 bits

def _exact_turn(case, x, seed_positions):
    """fp64 rows turned by complex multiplication."""
    rot = case["rot"]
    freqs, axis = _freqs(case).double().cuda(), torch.tensor(_axis_of_pairs(case), device="cuda")
    angle = seed_positions.double()[axis].permute(1, 2, 0) * freqs
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    y = x.double().clone()
    if case["pairs"] == "adjacent":
        z = torch.view_as_complex(y[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * turn
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot] = torch.cat([z.real, z.imag], dim=-1)
    return y


def _exact_quantised(x, codes):
    """The values that slabs x (fp64 of bf16, one scale for the last axis) are
    held as: the quotient is the fp32 one by definition."""
    scale = (x.abs().amax(-1, keepdim=True) / QMAX[codes]).float().double()
    y = torch.where(scale > 0, x / scale, 0.0).float().double()
    if codes == "e4m3":
        # 4 significant bits down to 2^-6, steps of 2^-9 below, at most 448
        step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(y / step) * step).clamp(-448.0, 448.0) * scale
    return torch.round(y).clamp(-127.0, 127.0) * scale


def _exact_held(case, x):
    """fp64 [..., tokens, 128] that the cache holds of whole sequences."""
    out = x.double()
    blocks = _closed(x.shape[-2], case["block"])
    end = SINKS + blocks * case["block"]
    body = _exact_quantised(out[..., SINKS:end, :].unflatten(-2, (blocks, -1)).flatten(-2), case["codes"]) \
        if blocks else out[..., SINKS:end, :]
    return torch.cat([out[..., :SINKS, :], body.reshape(*x.shape[:-2], -1, D), out[..., end:, :]], dim=-2)


def _exact_row(case, q, k, v, head, at, newest):
    """fp64 output of one query row over keys at positions `at`."""
    s = k @ q.double() / math.sqrt(D)
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    if case["bias"]:
        slope = float(torch.tensor(2.0 ** (-8.0 * (head + 1) / case["hq"]), dtype=torch.float32))
        s = s - slope * (newest - at).double()
    return torch.softmax(s, -1) @ v


def _exact_choice(case, q, k, closed):
    """Blocks that one KV head's query rows q [group, 128] choose among the
    closed blocks of keys k [tokens, 128]."""
    spare = max(closed - case["recent"], 0)
    if spare <= case["top"]:
        return list(range(closed))

    def eights(x, amax):
        scale = (amax / 127.0).float().double()
        return torch.where(scale > 0, x / scale, 0.0).float().double().round().clamp(-127, 127), scale

    body = k[SINKS:SINKS + closed * case["block"]].double().view(closed, case["block"], D)
    low, high = body.amin(1), body.amax(1)
    t = body.abs().amax((1, 2))[:, None]
    (low, _), (high, t) = eights(low, t), eights(high, t)
    best = torch.full((closed,), -math.inf, dtype=torch.float32, device="cuda")
    for row in q.double():
        code, s = eights(row, row.abs().max())
        bound = torch.maximum(code * low, code * high).sum(1)
        best = torch.maximum(best, ((bound * s).float().double() * t[:, 0]).float())
    score = best[:spare].tolist()
    order = sorted(range(spare), key=lambda c: (-score[c], c))[:case["top"]]
    return sorted(order) + list(range(spare, closed))


def exact(case, seed):
    if case["op"] in ("rotary", "append"):
        q, k, v = _draw_rows(case, seed)
        at = _positions(case)
        q, k = _exact_turn(case, q, at), _exact_turn(case, k, at)
        if case["op"] == "rotary":
            return q, k
        return q, _exact_held(case, k.to(torch.bfloat16)), _exact_held(case, v)
    q, kv = _draw_held(case, seed)
    group = case["hq"] // case["hkv"]
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    k, v, lengths = kv[-1]
    shared = case["prefix"] if case["op"] == "prefix" else 0
    most = case.get("top", 0) + case.get("recent", 0)
    chosen = torch.full((case["batch"], case["hkv"], most), -1, dtype=torch.int32, device="cuda")
    for h in range(case["hkv"]):
        front = [_exact_held(case, x[0, h]) for x in kv[0][:2]] if shared else None
        for b, n in enumerate(lengths):
            kd, vd = _exact_held(case, k[b, h, :n]), _exact_held(case, v[b, h, :n])
            at = torch.arange(shared + n, device="cuda")
            if shared:
                kd, vd = torch.cat([front[0], kd]), torch.cat([front[1], vd])
            else:
                closed = _closed(n, case["block"])
                blocks = _exact_choice(case, q[b, h * group:(h + 1) * group], k[b, h, :n], closed)
                chosen[b, h, :len(blocks)] = torch.tensor(blocks, dtype=torch.int32, device="cuda")
                keep = (at < SINKS) | (at >= SINKS + closed * case["block"])
                for c in blocks:
                    keep[SINKS + c * case["block"]:SINKS + (c + 1) * case["block"]] = True
                kd, vd, at = kd[keep], vd[keep], at[keep]
            for j in range(h * group, (h + 1) * group):
                out[b, j] = _exact_row(case, q[b, j], kd, vd, j, at, shared + n - 1)
    return out if shared else (out, chosen)
