"""The operators of a decoding step on low-bit weights and a low-bit cache: cases, inputs, plain forms.

Four groups of calls, named by a case's "op":
  matvec     imq_w4_matvec: a few tokens times a 4-bit weight with a step per group of inputs
  requant    imq_w4_quantize then imq_w4_dequantize: a weight brought to 4 bits, and the values it stands for
  cache      imq_kv_write then imq_kv_read: new keys and values quantised into a paged cache, a span read back
  attention  imq_paged_attention: one new token per sequence over the paged 8- or 4-bit cache

Quantisation (every group: a run of a weight's inputs, or one head's key or value vector of one token):
  q = max |x|, s = fp32(beta / q), step = fp32(q / beta), code = round_half_even(fp32(x * s)), where
  beta = 2^(bits - 1) - 1; a group with q = 0 has s = step = 1.  The value of a code is step * code.
Storage: code + 2^(bits - 1), one byte each at 8 bits; at 4 bits eight codes per 32-bit word, code e of the
eight in bits 4 * (e // 2 + 4 * (e % 2)) and up.  A weight row is cut into blocks of 128 inputs, 64 bytes
each; input r of a block belongs to word 4 * (r % 32 // 8) + r // 32 of the block's 16, as its code e = r % 8.
Cache pages are (page, head, token, bytes of a vector) for keys and for values, with the steps of both in
(page, head, token, 2).
"""
import math

import numpy as np
import torch

own = False

_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
# 4-bit codes e = 0..7 of a word, by the nibble that holds them
_NIBBLE_TO_CODE = (0, 2, 4, 6, 1, 3, 5, 7)


def listed():
    return [
        # one token through a 4096 x 4096 attention projection: the smallest common call, launch latency counts
        dict(name="matvec_proj_1", op="matvec", M=1, K=4096, N=4096, group=128, x="bf16", y="bf16"),
        # one token through the down projection (long inner axis), finer groups
        dict(name="matvec_down_1", op="matvec", M=1, K=11008, N=4096, group=64, x="bf16", y="bf16"),
        # eight sequences decoding at once through gate and up, stored as one weight
        dict(name="matvec_gate_up_8", op="matvec", M=8, K=4096, N=22016, group=128, x="bf16", y="bf16"),
        # fp32 activations, odd sizes, the finest groups
        dict(name="matvec_odd_3_f32", op="matvec", M=3, K=4099, N=11007, group=32, x="f32", y="f32"),
        # a projection's weight brought to 4 bits when a model is loaded
        dict(name="requant_proj", op="requant", K=4096, N=4096, group=128, x="bf16", trans=False),
        # an output-major fp32 weight of odd sizes
        dict(name="requant_odd_f32", op="requant", K=11003, N=4097, group=64, x="f32", trans=True),
        # a decoding step of 32 sequences: one key and value each, 8 bits; the same tokens read back
        dict(name="cache_step_8bit", op="cache", n=32, back=64, H=32, D=128, bits=8, page=16, x="bf16", y="bf16"),
        # a prompt's keys and values written at 4 bits, and a longer span read back for the next chunk
        dict(name="cache_prompt_4bit", op="cache", n=8191, back=12289, H=8, D=128, bits=4, page=64, x="bf16", y="f32"),
        # one sequence of 2048 tokens, 32 heads of 128 (the attention shape of this repository's workloads)
        dict(name="attention_1x2048", op="attention", B=1, Hq=32, H=32, D=128, bits=8, page=16, longest=2048, ragged=False,
             q="bf16", o="bf16"),
        # sixteen sequences of mixed lengths, four query heads to a key head, 4-bit cache
        dict(name="attention_16xmixed", op="attention", B=16, Hq=32, H=8, D=128, bits=4, page=64, longest=8192, ragged=True,
             q="bf16", o="bf16"),
        # one long context on few key heads: all the work is one sequence's length
        dict(name="attention_1x131072", op="attention", B=1, Hq=32, H=8, D=128, bits=8, page=64, longest=131072, ragged=False,
             q="bf16", o="bf16"),
        # a full serving batch, eight query heads to a key head, fp32 queries and outputs, some rows empty
        dict(name="attention_64xmixed_f32", op="attention", B=64, Hq=64, H=8, D=64, bits=8, page=32, longest=4097, ragged=True,
             q="f32", o="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("matvec", "requant", "cache", "attention", "matvec", "attention"))
    dt = lambda: rng.choice(("bf16", "bf16", "f32"))  # noqa: E731
    if op == "matvec":
        K = _log(rng, 64, 16384)
        N = _log(rng, 16, max(17, min(32768, 90_000_000 // K)))
        if rng.random() < 0.5:
            K, N = -(-K // 64) * 64, -(-N // 16) * 16
        return dict(op=op, M=_log(rng, 1, 16), K=K, N=N, group=rng.choice((32, 64, 128)), x=dt(), y=dt())
    if op == "requant":
        K = _log(rng, 64, 11008)
        return dict(op=op, K=K, N=_log(rng, 16, max(17, min(11008, 45_000_000 // K))), group=rng.choice((32, 64, 128)),
                    x=dt(), trans=rng.random() < 0.5)
    if op == "cache":
        H, D = rng.choice((1, 2, 4, 8, 16, 32)), rng.choice((64, 128, 192, 256))
        n = _log(rng, 1, max(2, min(8191, 8_000_000 // (H * D))))
        return dict(op=op, n=n, back=n + _log(rng, 1, n + 1), H=H, D=D, bits=rng.choice((4, 8)), page=rng.choice((16, 32, 48, 128)),
                    x=dt(), y=dt())
    B, H, D = _log(rng, 1, 64), rng.choice((1, 2, 4, 8, 32)), rng.choice((64, 128, 192, 256))
    most = max(16, min(131072, 120_000_000 // (B * H * D)))
    return dict(op=op, B=B, Hq=H * rng.choice((1, 2, 4, 7, 8, 16)), H=H, D=D, bits=rng.choice((4, 8)), page=rng.choice((16, 32, 48, 128)),
                longest=_log(rng, 1, most), ragged=rng.random() < 0.5, q=dt(), o=dt())


# ---------------------------------------------------------------------------------------------------------------
# quantisation and storage, in elementary operations
# ---------------------------------------------------------------------------------------------------------------
def _quantise(x, bits):
    """Codes (fp32 whole numbers) and steps of groups along the last axis."""
    q = x.float().abs().amax(-1)
    beta = torch.full_like(q, 2 ** (bits - 1) - 1)  # a tensor: a number's quotient would be a product with a reciprocal
    q = torch.where(q == 0, beta, q)  # s = step = 1
    return torch.round(x.float() * (beta / q).unsqueeze(-1)), q / beta


def _to_nibbles(codes):
    """(..., 8 n) codes of 4 bits as (..., 4 n) bytes."""
    u = (codes + 8).to(torch.int32).unflatten(-1, (-1, 8))[..., list(_NIBBLE_TO_CODE)].unflatten(-1, (4, 2))
    return (u[..., 0] + 16 * u[..., 1]).to(torch.uint8).flatten(-2)


def _from_nibbles(b):
    """(..., 4 n) bytes as (..., 8 n) fp32 codes."""
    u = torch.stack((b & 15, b >> 4), -1).unflatten(-2, (-1, 4)).flatten(-2)
    order = sorted(range(8), key=_NIBBLE_TO_CODE.__getitem__)
    return u[..., order].flatten(-2).float() - 8


def _pack_weight(codes):
    """(N, K) codes as (N, 64 * ceil(K / 128)) bytes in the weight's block order."""
    c = torch.nn.functional.pad(codes, (0, -codes.shape[1] % 128))
    return _to_nibbles(c.unflatten(1, (-1, 4, 4, 8)).transpose(2, 3).flatten(1)).contiguous()


def _unpack_weight(b, K):
    return _from_nibbles(b).unflatten(1, (-1, 4, 4, 8)).transpose(2, 3).flatten(1)[:, :K]


def _quantise_weight(W, group):
    """(N, K) values as fp32 codes (N, K) and steps (N, ceil(K / group)); the last group may be short."""
    K = W.shape[1]
    codes, steps = _quantise(torch.nn.functional.pad(W, (0, -K % group)).unflatten(1, (-1, group)), 4)
    return codes.flatten(1)[:, :K], steps


def _weight_values(codes, steps, group):
    return codes * steps.repeat_interleave(group, 1)[:, : codes.shape[1]]


def _pack_vectors(codes, bits):
    return _to_nibbles(codes) if bits == 4 else (codes + 128).to(torch.uint8)


def _unpack_vectors(b, bits):
    return _from_nibbles(b) if bits == 4 else b.float() - 128


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _vectors(g, n, H, D):
    """Keys or values as a model makes them: N(0, 1) with four heavy dimensions per head."""
    x = _normal(g, n, H, D)
    heavy = torch.rand(H, D, generator=g, device="cuda").argsort(-1)[:, :4]
    return x * torch.ones(H, D, device="cuda").scatter_(1, heavy, 20.0)


def _empty_cache(case, n_pages):
    H, page, D, bits = case["H"], case["page"], case["D"], case["bits"]
    k = torch.full((n_pages, H, page, D * bits // 8), 0x88 if bits == 4 else 0x80, dtype=torch.uint8, device="cuda")
    return {"k": k, "v": k.clone(), "steps": torch.ones(n_pages, H, page, 2, device="cuda")}


def _plain_write(s, k, v, slots):
    page, bits = s["case"]["page"], s["case"]["bits"]
    at, to = slots // page, slots % page
    kc, ks = _quantise(k, bits)
    vc, vs = _quantise(v, bits)
    s["k"][at, :, to] = _pack_vectors(kc, bits)
    s["v"][at, :, to] = _pack_vectors(vc, bits)
    s["steps"][at, :, to] = torch.stack((ks, vs), -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    if case["op"] in ("matvec", "requant"):
        # weights as this repository's linear layers have them: N(0, 0.02^2) with 0.05 % heavy entries
        K, N = case["K"], case["N"]
        W = _normal(g, N, K) * 0.02
        W = torch.where(torch.rand(N, K, generator=g, device="cuda") < 5e-4, W * 30, W).to(_DTYPE[case["x"]])
        if case["op"] == "requant":
            s["W"] = W if case["trans"] else W.t().contiguous()
        else:
            codes, steps = _quantise_weight(W, case["group"])
            s["codes"], s["steps"] = _pack_weight(codes), steps.contiguous()
            # activations: N(0, 1) with six heavy channels
            x = _normal(g, case["M"], K)
            x[:, torch.randperm(K, generator=g, device="cuda")[:6]] *= 60
            s["X"] = x.to(_DTYPE[case["x"]])
    elif case["op"] == "cache":
        n, back, page, dt = case["n"], case["back"], case["page"], _DTYPE[case["x"]]
        n_pages = -(-(back + 5) // page) + 1
        s.update(_empty_cache(case, n_pages))
        # positions 0 .. back - 1 of a sequence on shuffled pages; the last n of them are new
        pages = torch.randperm(n_pages, generator=g, device="cuda")
        t = torch.arange(back, device="cuda")
        s["back"] = pages[t // page] * page + t % page
        s["slots"] = s["back"][back - n:].contiguous()
        old = back - n
        _plain_write(s, _vectors(g, old, case["H"], case["D"]).to(dt), _vectors(g, old, case["H"], case["D"]).to(dt), s["back"][:old])
        s["new_k"], s["new_v"] = (_vectors(g, n, case["H"], case["D"]).to(dt) for _ in range(2))
    else:
        B, page, longest = case["B"], case["page"], case["longest"]
        width = -(-longest // page)
        lens = torch.full((B,), longest, device="cuda")
        if case["ragged"]:  # every eighth sequence has no token yet; one has the longest
            lens = (torch.rand(B, generator=g, device="cuda") * longest).long() + 1
            lens[::8] = 0
            lens[B // 2] = longest
        used = -(-lens // page)
        n_pages = int(used.sum()) + 1
        s.update(_empty_cache(case, n_pages))
        pages = torch.randperm(n_pages, generator=g, device="cuda")
        first = used.cumsum(0) - used
        j = torch.arange(width, device="cuda")
        at = pages[(first[:, None] + j).clamp(max=n_pages - 1)]
        s["table"] = torch.where(j < used[:, None], at, -torch.ones_like(at)).int().contiguous()
        s["lens"] = lens.int()
        total = n_pages * page
        slots = torch.arange(total, device="cuda")
        for lo in range(0, total, 16384):  # a part at a time: the values are made in fp32
            m = min(16384, total - lo)
            k, v = _vectors(g, m, case["H"], case["D"]), _vectors(g, m, case["H"], case["D"])
            _plain_write(s, k, v, slots[lo:lo + m])
        s["Q"] = _normal(g, B, case["Hq"], case["D"]).to(_DTYPE[case["q"]])
    if own:  # the handles a program keeps: the tensors above with their sizes
        import bit_integer_gemm_b200 as imq
        if case["op"] == "matvec":
            s["weight"] = imq.W4Weight(s["codes"], s["steps"], case["K"], case["N"], case["group"])
        elif case["op"] != "requant":
            s["cache"] = imq.KVCache(s["k"], s["v"], s["steps"], case["D"], case["bits"])
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def _plain(s):
    case = s["case"]
    if case["op"] == "matvec":
        W = _weight_values(_unpack_weight(s["codes"], case["K"]), s["steps"], case["group"])
        return (s["X"].float() @ W.t()).to(_DTYPE[case["y"]])
    if case["op"] == "requant":
        W = s["W"] if case["trans"] else s["W"].t()
        codes, steps = _quantise_weight(W, case["group"])
        values = _weight_values(_unpack_weight(_pack_weight(codes), case["K"]), steps, case["group"])
        values = values if case["trans"] else values.t().contiguous()
        return {"steps": steps, "values": values.to(_DTYPE[case["x"]])}
    page, bits = case["page"], case["bits"]
    if case["op"] == "cache":
        _plain_write(s, s["new_k"], s["new_v"], s["slots"])
        at, to = s["back"] // page, s["back"] % page
        steps = s["steps"][at, :, to]
        k = _unpack_vectors(s["k"][at, :, to], bits) * steps[..., :1]
        v = _unpack_vectors(s["v"][at, :, to], bits) * steps[..., 1:]
        return {"k": k.to(_DTYPE[case["y"]]), "v": v.to(_DTYPE[case["y"]]), "steps": s["steps"]}
    B, H, D, longest = case["B"], case["H"], case["D"], case["longest"]
    t = torch.arange(longest, device="cuda")
    at, to = s["table"].long().clamp(min=0)[:, t // page], t % page  # (B, t)
    steps = s["steps"][at, :, to]  # (B, t, H, 2)
    k = _unpack_vectors(s["k"][at, :, to], bits) * steps[..., :1]
    scores = torch.einsum("bhgd,bthd->bhgt", s["Q"].float().unflatten(1, (H, -1)), k) * (1 / math.sqrt(D))
    del k
    scores = scores.masked_fill(t >= s["lens"][:, None, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - top.clamp(min=torch.finfo(torch.float32).min)).exp()
    total = p.sum(-1, keepdim=True)
    v = _unpack_vectors(s["v"][at, :, to], bits) * steps[..., 1:]
    out = torch.einsum("bhgt,bthd->bhgd", p, v) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, top + total.log(), torch.full_like(top, -math.inf))
    return {"out": out.flatten(1, 2).to(_DTYPE[case["o"]]), "lse": lse.flatten(1)}


def run(state):
    if not own:
        return _plain(state)
    import bit_integer_gemm_b200 as imq
    case = state["case"]
    if case["op"] == "matvec":
        return imq.imq_w4_matvec(state["weight"], state["X"], out_dtype=_DTYPE[case["y"]])
    if case["op"] == "requant":
        w = imq.imq_w4_quantize(state["W"], case["group"], transW=case["trans"])
        return {"steps": w.steps, "values": imq.imq_w4_dequantize(w, _DTYPE[case["x"]], transW=case["trans"])}
    if case["op"] == "cache":
        imq.imq_kv_write(state["cache"], state["new_k"], state["new_v"], state["slots"])
        k, v = imq.imq_kv_read(state["cache"], state["back"], dtype=_DTYPE[case["y"]])
        return {"k": k, "v": v, "steps": state["steps"]}
    out, lse = imq.imq_paged_attention(state["cache"], state["Q"], state["table"], state["lens"], max_len=case["longest"],
                                       out_dtype=_DTYPE[case["o"]])
    return {"out": out, "lse": lse}


def _lengths(case):
    """The expected total length of an attention case (ragged lengths are uniform, one in eight empty)."""
    B, longest = case["B"], case["longest"]
    return B * longest if not case["ragged"] else (B - 1) * 7 / 8 * (longest + 1) / 2 + longest


def work(case):
    if case["op"] == "matvec":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": N * K / 2 + 4 * N * -(-K // case["group"]) + M * K * _SIZE[case["x"]] + M * N * _SIZE[case["y"]],
                "flops": 2.0 * M * N * K}
    if case["op"] == "requant":
        K, N = case["K"], case["N"]
        # quantised: the values in, codes and steps out; dequantised: codes and steps in, the values out
        return {"bytes": 2 * (N * K * (_SIZE[case["x"]] + 0.5) + 4 * N * -(-K // case["group"])), "flops": 4.0 * N * K}
    vector = 2 * (case["D"] * case["bits"] / 8 + 4)  # a key, a value and their steps
    if case["op"] == "cache":
        H, D, n, back = case["H"], case["D"], case["n"], case["back"]
        return {"bytes": n * (H * (2 * D * _SIZE[case["x"]] + vector) + 8) + back * (H * (2 * D * _SIZE[case["y"]] + vector) + 8),
                "flops": 4.0 * (n + back) * H * D}
    total, B, Hq, D = _lengths(case), case["B"], case["Hq"], case["D"]
    return {"bytes": total * (case["H"] * vector + 4 / case["page"]) + B * (Hq * (D * (_SIZE[case["q"]] + _SIZE[case["o"]]) + 4) + 4),
            "flops": 4.0 * total * Hq * D}


# ---------------------------------------------------------------------------------------------------------------
# the same in 64 bits, from the definitions, on the host where it is small and by sequence where it is not
# ---------------------------------------------------------------------------------------------------------------
def _exact_quantise(x, bits):
    """Codes and steps of fp64 groups (rows): each fp32 rounding of the definition taken from the 64-bit value
    (a quotient or product of two fp32 numbers rounded to 64 and then to 32 bits is the correctly rounded one)."""
    q = x.abs().max(dim=-1, keepdim=True).values
    beta = torch.full_like(q, 2.0 ** (bits - 1) - 1)
    s = torch.where(q > 0, beta / q, torch.ones_like(q)).float().double()
    step = torch.where(q > 0, q / beta, torch.ones_like(q)).float().double()
    return torch.round((x * s).float().double()), step


def _exact_bytes(b, bits):
    """Stored bytes (..., n) as fp64 codes, nibble by nibble."""
    if bits == 8:
        return b.double() - 128
    out = torch.empty(*b.shape[:-1], b.shape[-1] // 4, 8, dtype=torch.float64, device=b.device)
    w = b.reshape(*b.shape[:-1], -1, 4).long()
    for e in range(8):
        bit = 4 * (e // 2 + 4 * (e % 2))
        out[..., e] = ((w[..., bit // 8] >> (bit % 8)) & 15).double() - 8
    return out.flatten(-2)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "matvec":
        K, N, group = case["K"], case["N"], case["group"]
        r = np.arange(K)
        place = r // 128 * 128 + ((r % 32) // 8 * 4 + r % 128 // 32) * 8 + r % 8
        W = _exact_bytes(s["codes"], 4)[:, torch.from_numpy(place).cuda()]
        y = torch.zeros(case["M"], N, dtype=torch.float64, device="cuda")
        for i, lo in enumerate(range(0, K, group)):
            y += (s["X"][:, lo:lo + group].double() @ W[:, lo:lo + group].t()) * s["steps"][:, i].double()
        return y
    if case["op"] == "requant":
        W = (s["W"] if case["trans"] else s["W"].t()).double()
        steps, values = [], []
        for lo in range(0, case["K"], case["group"]):
            c, d = _exact_quantise(W[:, lo:lo + case["group"]], 4)
            steps.append(d)
            values.append(c * d)
        values = torch.cat(values, 1)
        return {"steps": torch.cat(steps, 1), "values": values if case["trans"] else values.t().contiguous()}
    page, bits, H = case["page"], case["bits"], case["H"]
    if case["op"] == "cache":
        old = case["back"] - case["n"]
        at, to = s["back"][:old] // page, s["back"][:old] % page
        got = {}
        for i, name in enumerate(("k", "v")):
            before = _exact_bytes(s[name][at, :, to], bits) * s["steps"][at, :, to, i, None].double()
            c, d = _exact_quantise(s["new_" + name].double(), bits)
            got[name] = torch.cat((before, c * d))
            s["steps"][s["slots"] // page, :, s["slots"] % page, i] = d[..., 0].float()
        return {**got, "steps": s["steps"].double()}
    B, Hq, D = case["B"], case["Hq"], case["D"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["lens"][b])
        if not n:
            continue
        pages = s["table"][b, : -(-n // page)].long()
        q = s["Q"][b].double().reshape(H, Hq // H, D)
        for h in range(H):
            steps = s["steps"][pages, h].double().reshape(-1, 2)[:n]
            k = _exact_bytes(s["k"][pages, h], bits).reshape(-1, D)[:n] * steps[:, :1]
            v = _exact_bytes(s["v"][pages, h], bits).reshape(-1, D)[:n] * steps[:, 1:]
            x = q[h] @ k.t() / math.sqrt(D)
            l = torch.logsumexp(x, -1)
            at = slice(h * (Hq // H), (h + 1) * (Hq // H))
            out[b, at], lse[b, at] = (x - l[:, None]).exp() @ v, l
    return {"out": out, "lse": lse}
