"""Timed cases of four operators of the compressed-KV library, each beside its
plain form in elementary torch operations.

decode   single-query attention over the per-token-scaled compressed cache
         (INT8, INT4 or FP8 E4M3 codes) whose scores are capped by a tanh
         and / or lowered by a slope per query head times the distance;
prompt   attention of a prompt over itself whose scores are capped or biased
         the same way, each query seeing one run of keys (causal, packed
         documents, a two-way prefix), with the column sums of its
         probabilities on request;
append   a prompt quantised into the block-scaled cache (one scale per block of
         tokens and KV head, the open block and the sinks in bf16) and read
         back as dense tensors;
attend   single-query attention over the block-scaled cache.

Definitions shared by all: 128 dims per head, query head j reads KV head
j / (Hq / Hkv); score = cap * tanh(s / cap) with s = q . k / sqrt(128) (s alone
where cap is 0), minus slope[j] * |query position - key position|.  The first
four positions of a sequence are kept in bf16.  Scale = amax / 127 (INT8),
amax / 7 (INT4) or amax / 448 (E4M3) in IEEE fp32, code = x / scale (IEEE fp32
division) rounded half to even.
"""
import math
import random

import torch

own = False

D = 128
SINKS = 4


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one chat sequence of a small model: the smallest call, all latency
        dict(name="decode_one_seq_int8_cap", op="decode", batch=1, hq=8, hkv=8, ctx=512, ragged=0, codes="int8",
             cap=50.0, bias=False),
        # a served batch of the 48-layer GQA stack's shape, INT4, distance bias
        dict(name="decode_gqa5_int4_bias", op="decode", batch=32, hq=40, hkv=8, ctx=8192, ragged=0, codes="int4",
             cap=0.0, bias=True),
        # a served batch with ragged contexts, FP8 codes, both transforms
        dict(name="decode_ragged_e4m3_cap_bias", op="decode", batch=16, hq=32, hkv=8, ctx=8192, ragged=11,
             codes="e4m3", cap=30.0, bias=True),
        # short packed documents, odd sizes: a small prefill
        dict(name="prompt_short_documents", op="prompt", batch=4, hq=8, hkv=2, n=517, layout=3, prefix=0, pads=1,
             cap=20.0, bias=False, sums=False),
        # one long prompt of a model with capped scores
        dict(name="prompt_long_causal_cap", op="prompt", batch=1, hq=32, hkv=8, n=8192, layout=0, prefix=0, pads=0,
             cap=50.0, bias=False, sums=False),
        # a long row of packed documents with a distance bias
        dict(name="prompt_packed_documents_bias", op="prompt", batch=1, hq=40, hkv=8, n=8000, layout=9, prefix=0,
             pads=1, cap=0.0, bias=True, sums=False),
        # prompts with a two-way prefix whose column sums seed an eviction
        dict(name="prompt_prefix_sums", op="prompt", batch=2, hq=32, hkv=32, n=2100, layout=0, prefix=700, pads=0,
             cap=30.0, bias=True, sums=True),
        # a short turn of many sequences
        dict(name="append_short_turns", op="append", batch=64, hkv=8, n=41, block=16, codes="int8"),
        # a batch of prompts of a model with 32 KV heads
        dict(name="append_prompts_int8", op="append", batch=16, hkv=32, n=4096, block=16, codes="int8"),
        # one block-scaled sequence: the smallest call
        dict(name="attend_one_seq", op="attend", batch=1, hq=8, hkv=8, ctx=517, ragged=0, block=16, codes="int8",
             cap=0.0, bias=False),
        # a served batch of a model with as many KV heads as query heads
        dict(name="attend_mha_int8_cap", op="attend", batch=16, hq=32, hkv=32, ctx=4111, ragged=0, block=32,
             codes="int8", cap=50.0, bias=False),
        # a few long ragged contexts, large blocks, FP8 codes, distance bias
        dict(name="attend_long_e4m3_bias", op="attend", batch=4, hq=32, hkv=8, ctx=32768, ragged=5, block=64,
             codes="e4m3", cap=0.0, bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "prompt", "append", "attend"])
    hkv = rng.choice([1, 2, 4, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8) if g * hkv <= 64])
    hq = hkv * group
    cap = rng.choice([0.0, round(rng.uniform(4.0, 60.0), 2)])
    bias = rng.random() < 0.5
    if op == "decode":
        ctx = _log_int(rng, 2, 32768)
        batch = _log_int(rng, 1, max(1, min(64, (1 << 21) // (ctx * hkv))))
        if cap == 0.0 and not bias:
            cap = 25.0
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, ctx=ctx, ragged=rng.choice([0, rng.randrange(1, 1000)]),
                    codes=rng.choice(["int8", "int4", "e4m3"]), cap=cap, bias=bias)
    if op == "prompt":
        two_way = rng.random() < 0.5
        most = 1.0e9 if two_way else 2.0e9
        n = _log_int(rng, 1, min(8000, int(math.sqrt(most / hq))))
        batch = _log_int(rng, 1, max(1, min(16, int(most / (float(n) * n * hq)))))
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, n=n, layout=rng.choice([0, rng.randrange(1, 1000)]),
                    prefix=rng.randrange(0, n + 1) if two_way else 0, pads=rng.choice([0, 1]), cap=cap, bias=bias,
                    sums=rng.random() < 0.5)
    if op == "append":
        n = _log_int(rng, 1, 16384)
        batch = _log_int(rng, 1, max(1, min(64, (1 << 21) // (n * hkv))))
        return dict(op=op, batch=batch, hkv=hkv, n=n, block=rng.choice([16, 32, 64, 128]),
                    codes=rng.choice(["int8", "e4m3"]))
    ctx = _log_int(rng, 1, 32768)
    batch = _log_int(rng, 1, max(1, min(64, (1 << 21) // (ctx * hkv))))
    return dict(op=op, batch=batch, hq=hq, hkv=hkv, ctx=ctx, ragged=rng.choice([0, rng.randrange(1, 1000)]),
                block=rng.choice([16, 32, 64, 128]), codes=rng.choice(["int8", "e4m3"]), cap=cap, bias=bias)


def _contexts(case):
    """Tokens held per sequence: all `ctx`, or spread over [ctx / 8, ctx]."""
    if not case["ragged"]:
        return [case["ctx"]] * case["batch"]
    r = random.Random(case["ragged"])
    return [r.randint(max(1, case["ctx"] // 8), case["ctx"]) for _ in range(case["batch"])]


def _runs(case):
    """(begin, end) of the keys that each query of a prompt row sees.

    layout 0: one document; else documents of random lengths packed end to
    end.  The first `prefix` tokens of each document see each other both
    ways.  With pads, the last few tokens are padding and see nothing.
    """
    n, r = case["n"], random.Random(case["layout"])
    cuts = [0]
    while cuts[-1] < n:
        left = n - cuts[-1]
        cuts.append(cuts[-1] + (left if not case["layout"] else min(left, r.randint(1, max(1, min(2500, n // 3))))))
    begin, end = [], []
    for a, b in zip(cuts, cuts[1:]):
        two_way = min(b, a + case["prefix"])
        begin += [a] * (b - a)
        end += [max(i + 1, two_way) if i < two_way else i + 1 for i in range(a, b)]
    if case["pads"]:
        for i in range(n - min(n // 8, 9), n):
            begin[i], end[i] = 0, 0
    return begin, end


def work(case):
    if case["op"] in ("decode", "attend"):
        tokens = sum(_contexts(case)) * case["hkv"]
        io = 2 * case["batch"] * case["hq"] * D * 2
        width = D // 2 if case["codes"] == "int4" else D
        per = 2 * width + (8 if case["op"] == "decode" else 8 / case["block"])
        return {"bytes": tokens * per + io, "flops": 4 * tokens * (case["hq"] // case["hkv"]) * D}
    if case["op"] == "prompt":
        begin, end = _runs(case)
        pairs = case["batch"] * case["hq"] * sum(e - b for b, e in zip(begin, end))
        rows = case["batch"] * case["n"] * D * 2
        sums = 4 * case["batch"] * case["hkv"] * case["n"] if case["sums"] else 0
        return {"bytes": rows * (2 * case["hq"] + 2 * case["hkv"]) + sums, "flops": 4 * pairs * D}
    values = 2 * case["batch"] * case["hkv"] * case["n"] * D
    return {"bytes": values * (2 + 1 + 1 + 2), "flops": 2 * values}


# -------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _keys(g, shape):
    """Keys with four outlier channels, as trained models have them."""
    k = torch.randn(shape, generator=g, device="cuda")
    k[..., torch.randperm(D, generator=g, device="cuda")[:4]] *= 6.0
    return k.to(torch.bfloat16)


def _slopes(case):
    """The geometric slopes of the distance bias."""
    if not case["bias"]:
        return None
    return torch.tensor([2.0 ** (-8.0 * (j + 1) / case["hq"]) for j in range(case["hq"])], device="cuda")


QMAX = {"int8": 127.0, "int4": 7.0, "e4m3": 448.0}


def _codes(x, amax, codes):
    """(codes, scale) of fp32 values x whose largest magnitude is amax."""
    scale = amax / torch.full_like(amax, QMAX[codes])
    y = torch.where(scale > 0, x / scale, torch.zeros_like(x))
    if codes == "e4m3":
        return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale
    low = -8.0 if codes == "int4" else -127.0
    return y.round().clamp(low, QMAX[codes]).to(torch.int8), scale


def _draw_inputs(case, seed):
    """q, k, v (bf16) of a case."""
    g = _generator(seed)
    n = case["ctx"] if case["op"] in ("decode", "attend") else case["n"]
    k = _keys(g, (case["batch"], case["hkv"], n, D))
    v = torch.randn((case["batch"], case["hkv"], n, D), generator=g, device="cuda").to(torch.bfloat16)
    q = None
    if case["op"] in ("decode", "attend"):
        q = torch.randn((case["batch"], case["hq"], D), generator=g, device="cuda").to(torch.bfloat16)
    elif case["op"] == "prompt":
        q = torch.randn((case["batch"], case["hq"], n, D), generator=g, device="cuda").to(torch.bfloat16)
    return q, k, v


def prepare(case, seed):
    q, k, v = _draw_inputs(case, seed)
    state = dict(case=case, q=q)
    if case["op"] in ("decode", "attend", "prompt"):
        state["slopes"] = _slopes(case)
    if case["op"] == "prompt":
        begin, end = _runs(case)
        rows = torch.tensor([begin, end], dtype=torch.int32, device="cuda")
        state |= dict(k=k, v=v, begin=rows[0].expand(case["batch"], -1).contiguous(),
                      end=rows[1].expand(case["batch"], -1).contiguous(),
                      status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        return state
    if case["op"] == "append":
        state |= dict(k=k, v=v)
        if own:
            from compressed_kv_cache_kvc_gb300 import BlockScaledCache
            per_seq = case["n"] // case["block"] + 1
            state["cache"] = BlockScaledCache(case["hkv"], case["hkv"], case["batch"] * per_seq, case["batch"],
                                              per_seq, block_tokens=case["block"], codes=case["codes"])
        return state
    lens = _contexts(case)
    state["lens"] = torch.tensor(lens, device="cuda")
    if own:
        from compressed_kv_cache_kvc_gb300 import BlockScaledCache, KVCache
        if case["op"] == "decode":
            per_seq = case["ctx"] // 16 + 1
            cache = KVCache(case["hq"], case["hkv"], 4 if case["codes"] == "int4" else 8, case["batch"] * per_seq,
                            case["batch"], per_seq, codes="e4m3" if case["codes"] == "e4m3" else "int")
            cache.set_score_transform(softcap=case["cap"], slopes=state["slopes"])
            append = cache.quantize_append
        else:
            per_seq = case["ctx"] // case["block"] + 1
            cache = BlockScaledCache(case["hq"], case["hkv"], case["batch"] * per_seq, case["batch"], per_seq,
                                     block_tokens=case["block"], codes=case["codes"])
            append = cache.append
        if case["ragged"]:
            for b, n in enumerate(lens):
                append(k[b:b + 1, :, :n].contiguous(), v[b:b + 1, :, :n].contiguous(), seq_begin=b)
        else:
            append(k, v)
        state["cache"] = cache
        return state
    # the plain form's cache: codes of every position (those of exact positions
    # are not used), scales, and the exact rows with their positions
    at = torch.arange(case["ctx"], device="cuda")
    for name, x in (("k", k.float()), ("v", v.float())):
        if case["op"] == "decode":
            c, s = _codes(x, x.abs().amax(-1, keepdim=True), case["codes"])
        else:
            block = case["block"]
            body = max(case["ctx"] - SINKS, 0)
            blocks = -(-body // block)
            x = torch.nn.functional.pad(x[:, :, SINKS:], (0, 0, 0, blocks * block - body))
            x = x.reshape(case["batch"], case["hkv"], blocks, block, D)
            c, s = _codes(x, x.abs().amax((-1, -2), keepdim=True), case["codes"])
        state[name + "_codes"], state[name + "_scale"] = c, s
    if case["op"] == "decode":
        exact = (at < SINKS).expand(case["batch"], -1)
    else:
        closed = SINKS + (state["lens"] - SINKS).clamp(min=0) // case["block"] * case["block"]
        exact = (at < SINKS) | ((at >= closed[:, None]) & (at < state["lens"][:, None]))
    b, t = exact.nonzero(as_tuple=True)
    state |= dict(exact_b=b, exact_t=t, k_exact=k[b, :, t], v_exact=v[b, :, t])
    return state


# --------------------------------------------------------------- plain forms

def _dense(state, name):
    """fp32 [batch, hkv, ctx, 128] of the plain form's cache."""
    case, x = state["case"], state[name + "_codes"].float()
    x = x * state[name + "_scale"]
    if case["op"] == "attend":
        x = x.flatten(2, 3)
        x = torch.nn.functional.pad(x, (0, 0, SINKS, 0))[:, :, :case["ctx"]]
    x[state["exact_b"], :, state["exact_t"]] = state[name + "_exact"].float()
    return x


def _transform(s, case, slopes, distance):
    """Scores s (fp32 [batch, hkv, group, rows, keys]), capped and biased."""
    if case["cap"]:
        s = torch.tanh(s / case["cap"]) * case["cap"]
    if slopes is not None:
        s = s - slopes.view(case["hkv"], -1, 1, 1) * distance
    return s


def _softmax_product(s, seen, v):
    """(probabilities, probabilities . v), rows that see nothing being 0."""
    s = s.masked_fill_(~seen, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    return p, p @ v.unsqueeze(2)


def _plain_attention(state):
    case = state["case"]
    k, v = _dense(state, "k"), _dense(state, "v")
    q = state["q"].float().view(case["batch"], case["hkv"], -1, 1, D)
    s = (q @ k.unsqueeze(2).transpose(-1, -2)) * (1.0 / math.sqrt(D))
    at = torch.arange(case["ctx"], device="cuda")
    lens = state["lens"].view(-1, 1, 1, 1, 1)
    s = _transform(s, case, state["slopes"], (lens - 1 - at).float())
    out = _softmax_product(s, at < lens, v)[1]
    return out.reshape(case["batch"], case["hq"], D).to(torch.bfloat16)


def _plain_prompt(state):
    case = state["case"]
    n = case["n"]
    q = state["q"].float().view(case["batch"], case["hkv"], -1, n, D)
    k, v = state["k"].float(), state["v"].float()
    s = (q @ k.unsqueeze(2).transpose(-1, -2)) * (1.0 / math.sqrt(D))
    at = torch.arange(n, device="cuda")
    s = _transform(s, case, state["slopes"], (at[:, None] - at).abs().float())
    begin, end = (state[x].view(-1, 1, 1, n, 1) for x in ("begin", "end"))
    p, out = _softmax_product(s, (at >= begin) & (at < end), v)
    out = out.reshape(case["batch"], case["hq"], n, D).to(torch.bfloat16)
    if not case["sums"]:
        return out
    return out, p.sum((2, 3), dtype=torch.float64).float()


def _plain_append(state):
    case, got = state["case"], []
    block, n = case["block"], case["n"]
    blocks = max(n - SINKS, 0) // block

    def read(t):
        x = t[:, :, SINKS:SINKS + blocks * block].float().reshape(case["batch"], case["hkv"], blocks, block, D)
        if blocks:
            c, scale = _codes(x, x.abs().amax((-1, -2), keepdim=True), case["codes"])
            x = c.float() * scale
        x = x.reshape(case["batch"], case["hkv"], blocks * block, D).to(torch.bfloat16)
        return torch.cat([t[:, :, :SINKS], x, t[:, :, SINKS + blocks * block:]], dim=2)

    return read(state["k"]), read(state["v"])


# ----------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if not own:
        return {"decode": _plain_attention, "attend": _plain_attention, "prompt": _plain_prompt,
                "append": _plain_append}[case["op"]](state)
    if case["op"] == "decode":
        return state["cache"].decode_attention(state["q"], accumulate_h2o=False)
    if case["op"] == "attend":
        return state["cache"].decode_attention(state["q"], softcap=case["cap"], slopes=state["slopes"])
    if case["op"] == "append":
        cache = state["cache"]
        cache.release(0, case["batch"])
        cache.append(state["k"], state["v"])
        return cache.read(0, case["batch"], 0, case["n"])
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    return prompt_attention(state["q"], state["k"], state["v"], status=state["status"], softcap=case["cap"],
                            slopes=state["slopes"], key_begin=state["begin"], key_end=state["end"],
                            column_sums=case["sums"])


# -------------------------------------------------------------- in 64 bits

def _exact_quantised(x, codes):
    """The values that a slab x (fp64 of bf16, one scale for the whole last
    axis) is held as: the quotient is the fp32 one by definition."""
    scale = (x.abs().amax(-1, keepdim=True) / QMAX[codes]).float().double()
    y = torch.where(scale > 0, x / scale, 0.0).float().double()
    if codes == "e4m3":
        # 4 significant bits down to 2^-6, steps of 2^-9 below, at most 448
        step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        y = torch.round(y / step) * step
        y = y.clamp(-448.0, 448.0)
    else:
        y = torch.round(y).clamp(-8.0 if codes == "int4" else -127.0, QMAX[codes])
    return y * scale


def _exact_held(case, x, length):
    """fp64 [tokens, 128] that the cache holds for one sequence and head."""
    x = x[:length].double()
    out = x.clone()
    if case["op"] == "decode":
        out[SINKS:] = _exact_quantised(x[SINKS:], case["codes"])
        return out
    blocks = max(length - SINKS, 0) // case["block"]
    body = x[SINKS:SINKS + blocks * case["block"]]
    if blocks:
        out[SINKS:SINKS + body.shape[0]] = _exact_quantised(body.reshape(blocks, -1), case["codes"]).reshape(-1, D)
    return out


def _exact_rows(case, q, k, v, head, rows, begin, end):
    """fp64 probabilities and outputs of query rows at positions `rows`."""
    s = q.double() @ k.T / math.sqrt(D)
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    at = torch.arange(k.shape[0], device="cuda")
    if case["bias"]:
        slope = float(torch.tensor(2.0 ** (-8.0 * (head + 1) / case["hq"]), dtype=torch.float32))
        s = s - slope * (rows[:, None] - at).abs().double()
    s = torch.where((at >= begin[:, None]) & (at < end[:, None]), s, -math.inf)
    p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
    return p, p @ v


def exact(case, seed):
    q, k, v = _draw_inputs(case, seed)
    group = case["hq"] // case["hkv"] if "hq" in case else 1
    if case["op"] == "append":
        return [torch.stack([torch.stack([_exact_held(case, x[b, h], case["n"]) for h in range(case["hkv"])])
                             for b in range(case["batch"])]) for x in (k, v)]
    if case["op"] == "prompt":
        n = case["n"]
        begin, end = (torch.tensor(x, device="cuda") for x in _runs(case))
        rows = torch.arange(n, device="cuda")
        out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        sums = torch.zeros((case["batch"], case["hkv"], n), dtype=torch.float64, device="cuda")
        for b in range(case["batch"]):
            for j in range(case["hq"]):
                h = j // group
                p, out[b, j] = _exact_rows(case, q[b, j], k[b, h].double(), v[b, h].double(), j, rows, begin, end)
                sums[b, h] += p.sum(0)
        return (out, sums) if case["sums"] else out
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(_contexts(case)):
        last = torch.tensor([length - 1], device="cuda")
        for h in range(case["hkv"]):
            kd, vd = _exact_held(case, k[b, h], length), _exact_held(case, v[b, h], length)
            for j in range(h * group, (h + 1) * group):
                out[b, j] = _exact_rows(case, q[b, j:j + 1], kd, vd, j, last, 0 * last, last + 1)[1][0]
    return out
