"""Measured cases of the serving operators around the paged latent decode.

Each case is one pass through one operator: rotary positions, the cache write (bf16 and
FP8), the cache read-back, the FP8 decode for more than 16 query rows per latent head, and
the verification of drafted tokens.  ``own`` selects the library's kernels; otherwise the
same operator is computed from elementary torch operations.
"""

import math

import numpy as np
import torch

own = False

PAGE, D, DV, ROPE = 64, 576, 512, 64
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------- the cases
def listed():
    return [
        # rotary positions of the decode step's query heads: the rope columns of the [T, H, 192]
        # query projection (128 tokens x 128 heads, the shape of the absorption products)
        dict(name="rope step", op="rope", tokens=128, heads=128, width=64, row=192, rot=64, interleaved=True,
             inverse=False, factor=40.0, far=131072, dtype="bf16"),
        # a prompt's queries, positional part behind 128 columns that pass through; half layout
        dict(name="rope prompt", op="rope", tokens=4093, heads=128, width=192, row=192, rot=64, interleaved=False,
             inverse=False, factor=4.0, far=16384, dtype="bf16"),
        # the gradient's direction, fp32, few heads, unscaled frequencies
        dict(name="rope back fp32", op="rope", tokens=2049, heads=16, width=64, row=64, rot=64, interleaved=True,
             inverse=True, factor=1.0, far=4096, dtype="fp32"),
        # the step's new tokens into the cache: 64 sequences of the memory-bound decode, one token each
        dict(name="write step bf16", op="write", tokens=64, h_kv=1, fp8=False, norm=True, interleaved=True,
             far=4096, spare=1.0),
        # 32 sequences x 2 tokens of the multi-token decode into the FP8 cache
        dict(name="write step fp8", op="write", tokens=64, h_kv=1, fp8=True, norm=True, interleaved=True,
             far=16384, spare=1.0),
        # a long prompt into the FP8 cache
        dict(name="write prompt fp8", op="write", tokens=65521, h_kv=1, fp8=True, norm=True, interleaved=False,
             far=65536, spare=0.05),
        # a cached prefix of 16 sequences read back for the next prompt chunk, bf16
        dict(name="read prefix bf16", op="read", tokens=7777, h_kv=1, fp8=False, spare=0.5),
        # one 65,536-token sequence read back from the FP8 cache
        dict(name="read long fp8", op="read", tokens=65521, h_kv=1, fp8=True, spare=0.05),
        # the compute-bound decode (128 sequences x 128 heads x 4,096 tokens) over the FP8 cache
        dict(name="decode fp8 128 rows", op="decode", batch=128, s_q=1, h_q=128, h_kv=1, lo=4096, hi=4096, causal=True),
        # two tokens per sequence, 64 heads, ragged lengths from one token on
        dict(name="decode fp8 ragged", op="decode", batch=33, s_q=2, h_q=64, h_kv=1, lo=1, hi=8191, causal=True),
        # three drafted tokens for 64 sequences, fp32 probabilities over 131,072 tokens
        dict(name="verify batch", op="verify", batch=64, drafts=3, vocab=131072, dtype="fp32", greedy_draft=False),
        # one sequence, one deterministic draft, bf16 probabilities, odd vocabulary
        dict(name="verify one", op="verify", batch=1, drafts=1, vocab=32003, dtype="bf16", greedy_draft=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "decode", "verify"])
    if op == "rope":
        tokens, heads = _log(rng, 1, 16384), rng.choice([1, 8, 16, 64, 128])
        tokens = min(tokens, 500000 // heads)
        rot = rng.choice([32, 64, 64, 64, 128])
        width = rot + rng.choice([0, 0, 128])
        return dict(op=op, tokens=tokens, heads=heads, width=width, row=width + rng.choice([0, 8, 128]), rot=rot,
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.3,
                    factor=rng.choice([1.0, 4.0, 40.0]), far=_log(rng, 16, 1 << 20),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 50000), h_kv=rng.choice([1, 1, 1, 2]),
                    fp8=rng.random() < 0.5, norm=rng.random() < 0.7, interleaved=rng.random() < 0.5,
                    far=_log(rng, 16, 1 << 20), spare=rng.choice([0.05, 0.5, 1.0]))
    if op == "read":
        return dict(op=op, tokens=_log(rng, 1, 50000), h_kv=rng.choice([1, 1, 2]), fp8=rng.random() < 0.5,
                    spare=rng.choice([0.05, 0.5, 1.0]))
    if op == "decode":
        s_q = rng.choice([1, 1, 2, 3])
        h_kv = rng.choice([1, 1, 1, 2])
        g = rng.choice([24, 32, 64, 64, 128])
        hi = _log(rng, 8, 16384)
        batch = _log(rng, 1, max(2, min(128, 262144 // hi // h_kv)))
        return dict(op=op, batch=batch, s_q=s_q, h_q=g * h_kv, h_kv=h_kv, lo=rng.choice([0, 1, hi]), hi=hi,
                    causal=rng.random() < 0.7)
    return dict(op="verify", batch=_log(rng, 1, 48), drafts=rng.choice([1, 2, 3, 5, 8]), vocab=_log(rng, 1000, 131072),
                dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), greedy_draft=rng.random() < 0.25)


# ---------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _frequencies(rot, factor, base=10000.0, original=4096, fast=32.0, slow=1.0):
    """Rotary frequencies base^(-2i/rot); for factor > 1 the slow ones are divided by it and the
    ones in between blended over the pairs that turn `slow` to `fast` times in `original` tokens."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    if factor == 1.0:
        return f
    turn = [rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow)]
    low, high = max(math.floor(turn[0]), 0), min(math.ceil(turn[1]), rot - 1)
    ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp)


def _normal(shape, g, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _lengths(case, g):
    """Lengths spread evenly from hi down to lo, in an order of the seed's own."""
    n = torch.linspace(case["hi"], case["lo"], case["batch"], dtype=torch.float64).round().to(torch.int32).cuda()
    return n[torch.randperm(case["batch"], generator=g, device="cuda")]


def _codes(rows):
    amax = rows.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (rows / scale[..., None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = _gen(seed)
    op, c = case["op"], dict(case)
    if op == "rope":
        x = _normal((case["tokens"], case["heads"], case["row"]), g, _TYPES[case["dtype"]])
        c["x"] = x[..., case["row"] - case["width"]:]
        c["pos"] = torch.randint(0, case["far"], (case["tokens"],), generator=g, device="cuda")
        c["freq"] = _frequencies(case["rot"], case["factor"]).cuda()
        c["mag"] = 0.1 * math.log(case["factor"]) + 1.0
    elif op in ("write", "read"):
        t, h = case["tokens"], case["h_kv"]
        pages = -(-int(t * (1 + case["spare"])) // PAGE) + 1
        c["slots"] = torch.randperm(pages * PAGE, generator=g, device="cuda")[:t]
        if op == "read" or not case["fp8"]:
            c["pool"] = _normal((pages, PAGE, h, D), g, torch.bfloat16)
        if case["fp8"]:
            if op == "read":
                codes, scale = _codes(c.pop("pool").float())
                c["k8"], c["scale"] = codes, scale.permute(2, 0, 1).contiguous()
            else:
                c["k8"] = torch.zeros((pages, PAGE, h, D), dtype=torch.float8_e4m3fn, device="cuda")
                c["scale"] = torch.ones((h, pages, PAGE), device="cuda")
        if op == "write":
            # one projection's output, latent columns then rope columns, as a model produces it
            both = _normal((t, h, D), g, torch.bfloat16, 2.0)
            c["latent"], c["rope"] = both[..., :DV], both[..., DV:]
            c["weight"] = (1 + _normal((DV,), g, std=0.1)).to(torch.bfloat16) if case["norm"] else None
            c["pos"] = torch.randint(0, case["far"], (t,), generator=g, device="cuda").to(torch.int32)
            c["freq"] = _frequencies(ROPE, 40.0).cuda()
            c["mag"] = 1.0
    elif op == "decode":
        b, h = case["batch"], case["h_kv"]
        c["lens"] = _lengths(case, g)
        width = max(1, -(-case["hi"] // PAGE))
        pages = b * width
        rows = _normal((pages, PAGE, h, D), g, torch.bfloat16)
        rows[torch.rand((pages, PAGE), generator=g, device="cuda") < 0.05] *= 8  # outlier tokens
        codes, scale = _codes(rows.float())
        c["k8"], c["scale"] = codes, scale.permute(2, 0, 1).contiguous()
        c["table"] = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(b, width)
        c["q"] = _normal((b, case["s_q"], case["h_q"], D), g, torch.bfloat16)
    else:
        b, s, v = case["batch"], case["drafts"], case["vocab"]
        t = _TYPES[case["dtype"]]
        logits = _normal((b, s + 1, v), g, std=3.0)
        target = torch.softmax(logits, -1)
        if case["greedy_draft"]:
            c["draft"] = None
            c["tokens"] = target[:, :s].argmax(-1).to(torch.int32)
        else:
            draft = torch.softmax(logits[:, :s] + _normal((b, s, v), g, std=0.6), -1)
            c["tokens"] = torch.multinomial(draft.view(b * s, v), 1, generator=g).view(b, s).to(torch.int32)
            c["draft"] = draft.to(t)
        c["target"] = target.to(t)
        c["u"] = torch.rand((b, s), generator=g, device="cuda")
        c["u_new"] = torch.rand((b,), generator=g, device="cuda")
        c["n"] = torch.randint(0, s + 1, (b,), generator=g, device="cuda").to(torch.int32) if s > 1 else \
            torch.full((b,), s, dtype=torch.int32, device="cuda")
    return c


# ---------------------------------------------------------------------------- plain forms
def _rotate(x, pos, freq, interleaved, magnitude, inverse=False):
    """x [..., T, H, 2n] in fp32, angles in fp64."""
    n = freq.numel()
    a = pos.double()[:, None] * freq
    cos, sin = (a.cos() * magnitude).float()[:, None], (a.sin() * magnitude).float()[:, None]
    if inverse:
        sin = -sin
    x0, x1 = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :n], x[..., n:])
    y0, y1 = x0 * cos - x1 * sin, x0 * sin + x1 * cos
    return torch.stack((y0, y1), -1).flatten(-2) if interleaved else torch.cat((y0, y1), -1)


def _plain_rope(s):
    x, rot = s["x"], s["rot"]
    y = _rotate(x[..., s["width"] - rot:].float(), s["pos"], s["freq"], s["interleaved"], s["mag"], s["inverse"])
    return torch.cat((x[..., :s["width"] - rot], y.to(x.dtype)), -1)


def _plain_write(s):
    lat = s["latent"].float()
    if s["weight"] is not None:
        lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    row = torch.cat((lat, _rotate(s["rope"].float(), s["pos"], s["freq"], s["interleaved"], s["mag"])), -1)
    if not s["fp8"]:
        s["pool"].view(-1, s["h_kv"], D)[s["slots"]] = row.to(torch.bfloat16)
        return s["pool"]
    codes, scale = _codes(row)
    s["k8"].view(torch.uint8).view(-1, s["h_kv"], D)[s["slots"]] = codes.view(torch.uint8)
    s["scale"].view(s["h_kv"], -1)[:, s["slots"]] = scale.t()
    return s["k8"], s["scale"]


def _plain_read(s):
    if not s["fp8"]:
        return s["pool"].view(-1, s["h_kv"], D)[s["slots"]]
    codes = s["k8"].view(torch.uint8).view(-1, s["h_kv"], D)[s["slots"]].view(torch.float8_e4m3fn).float()
    return (codes * s["scale"].view(s["h_kv"], -1)[:, s["slots"]].t()[..., None]).to(torch.bfloat16)


def _plain_decode(s):
    b, s_q, h_q, h = s["batch"], s["s_q"], s["h_q"], s["h_kv"]
    table = s["table"].long()
    keys = s["k8"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * s["scale"][:, table].permute(1, 2, 3, 0)[..., None]
    keys = keys.flatten(1, 2).transpose(1, 2)                                # [b, h, n, 576]
    q = s["q"].float().view(b, s_q, h, h_q // h, D).transpose(1, 2).flatten(2, 3)  # [b, h, s_q * g, 576]
    x = torch.matmul(q, keys.transpose(-1, -2)).view(b, h, s_q, h_q // h, -1) * D ** -0.5
    at = torch.arange(x.shape[-1], device="cuda")
    back = torch.arange(s_q - 1, -1, -1, device="cuda") if s["causal"] else torch.zeros(s_q, dtype=torch.int64, device="cuda")
    seen = at < (s["lens"].long()[:, None] - back)[..., None]                # [b, s_q, n]
    x = x.masked_fill(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min(-1e30)
    e = (x - top).exp()
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e.flatten(2, 3), keys[..., :DV]).view(b, h, s_q, h_q // h, DV) / z.clamp_min(1e-30)
    lse = torch.where(z > 0, top + z.log(), -math.inf).squeeze(-1)
    return o.permute(0, 2, 1, 3, 4).reshape(b, s_q, h_q, DV).to(torch.bfloat16), lse.permute(0, 1, 3, 2).reshape(b, h_q, s_q)


def _plain_verify(s):
    b, k, v = s["batch"], s["drafts"], s["vocab"]
    target, draft, tokens = s["target"], s["draft"], s["tokens"].long()
    p = target[:, :k].gather(2, tokens[..., None]).squeeze(-1).double()
    q = draft.gather(2, tokens[..., None]).squeeze(-1).double() if draft is not None else torch.ones_like(p)
    place = torch.arange(k, device="cuda")
    good = (s["u"].double() * q < p) & (place < s["n"].long()[:, None])
    count = good.long().cumprod(1).sum(1)
    seq = torch.arange(b, device="cuda")
    w = target[seq, count].double()
    last = count.clamp_max(k - 1)
    less = draft[seq, last].double() if draft is not None else \
        torch.zeros_like(w).scatter_(1, tokens[seq, last][:, None], 1.0)
    rest = (w - less).clamp_min(0)
    use = (count < s["n"]) & (rest.sum(1) > 0)
    w = torch.where(use[:, None], rest, w)
    c = w.cumsum(1)
    over = c > (s["u_new"].double() * w.sum(1))[:, None]
    ids = torch.arange(v, device="cuda")
    new = torch.where(over.any(1), over.long().argmax(1), torch.where(w > 0, ids, -1).amax(1))
    out = torch.full((b, k + 1), -1, dtype=torch.int64, device="cuda")
    out[:, :k] = torch.where(place < count[:, None], tokens, -1)
    out[seq, count] = new
    return count.to(torch.int32), out.to(torch.int32)


_PLAIN = dict(rope=_plain_rope, write=_plain_write, read=_plain_read, decode=_plain_decode, verify=_plain_verify)


# ---------------------------------------------------------------------------- the library's calls
def _own(s):
    from paged_mla_decode_11_b200 import ops
    op = s["op"]
    if op == "rope":
        return ops.mla_rope(s["x"], s["pos"], s["freq"], interleaved=s["interleaved"], magnitude=s["mag"],
                            inverse=s["inverse"])
    if op == "write":
        how = dict(norm_weight=s["weight"], eps=1e-6, positions=s["pos"], inv_freq=s["freq"],
                   interleaved=s["interleaved"], magnitude=s["mag"])
        if not s["fp8"]:
            ops.mla_cache_write(s["latent"], s["rope"], s["slots"], s["pool"], **how)
            return s["pool"]
        ops.mla_cache_write_fp8(s["latent"], s["rope"], s["slots"], s["k8"], s["scale"], **how)
        return s["k8"], s["scale"]
    if op == "read":
        if s["fp8"]:
            return ops.mla_cache_read_fp8(s["k8"], s["scale"], s["slots"])
        return ops.mla_cache_read(s["pool"], s["slots"])
    if op == "decode":
        plan, splits = ops.get_mla_metadata(s["lens"], s["s_q"] * s["h_q"] // s["h_kv"], s["h_kv"])
        return ops.mla_decode_paged_fp8_rows(s["q"], s["k8"], s["scale"], s["table"], s["lens"], DV, plan, splits,
                                             causal=s["causal"])
    return ops.mla_verify_draft(s["target"], s["tokens"], s["u"], s["u_new"], draft_probs=s["draft"],
                                num_drafts=s["n"])


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------- work and exact values
def work(case):
    op = case["op"]
    if op == "rope":
        n, size = case["tokens"] * case["heads"], 4 if case["dtype"] == "fp32" else 2
        return dict(bytes=2 * n * case["width"] * size + 8 * case["tokens"], flops=3 * n * case["rot"])
    if op == "write":
        rows = case["tokens"] * case["h_kv"]
        return dict(bytes=rows * (2 * D + (D + 4 if case["fp8"] else 2 * D)) + 12 * case["tokens"],
                    flops=rows * (4 * DV + 3 * ROPE))
    if op == "read":
        rows = case["tokens"] * case["h_kv"]
        return dict(bytes=rows * (2 * D + (D + 4 if case["fp8"] else 2 * D)) + 8 * case["tokens"], flops=rows * D)
    if op == "decode":
        lens = np.round(np.linspace(case["hi"], case["lo"], case["batch"]))
        rows = case["batch"] * case["s_q"] * case["h_q"]
        seen = sum(np.maximum(lens - (i if case["causal"] else 0), 0).sum() for i in range(case["s_q"]))
        return dict(bytes=float(lens.sum() * case["h_kv"] * (D + 4) + rows * (2 * D + 2 * DV + 4)),
                    flops=float(seen * case["h_q"] * 2 * (D + DV)))
    # the row that is sampled from, and the draft's beside it where a draft was rejected
    size = 4 if case["dtype"] == "fp32" else 2
    rows = 1 if case["greedy_draft"] else 1.5
    return dict(bytes=case["batch"] * rows * case["vocab"] * size, flops=case["batch"] * 4 * case["vocab"])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def turned(x, mag, back):
        """The rotation as a product of complex numbers."""
        n = s["freq"].numel()
        z = torch.complex(x[..., 0::2], x[..., 1::2]) if s["interleaved"] else torch.complex(x[..., :n], x[..., n:])
        a = s["pos"].to(torch.float64).outer(s["freq"])[:, None, :]
        z = z * torch.polar(torch.full_like(a, mag), -a if back else a)
        y = torch.empty_like(x)
        if s["interleaved"]:
            y[..., 0::2], y[..., 1::2] = z.real, z.imag
        else:
            y[..., :n], y[..., n:] = z.real, z.imag
        return y

    if op == "rope":
        y = s["x"].double().clone()
        y[..., case["width"] - case["rot"]:] = turned(y[..., case["width"] - case["rot"]:].contiguous(), s["mag"], s["inverse"])
        return y
    if op == "write":
        row = torch.empty((case["tokens"], case["h_kv"], D), dtype=torch.float64, device="cuda")
        row[..., DV:] = turned(s["rope"].double().contiguous(), s["mag"], False)
        row[..., :DV] = s["latent"].double()
        if s["weight"] is not None:
            norm = torch.linalg.vector_norm(row[..., :DV], dim=-1, keepdim=True)
            row[..., :DV] *= s["weight"].double() / torch.sqrt(norm ** 2 / DV + 1e-6)
        if not case["fp8"]:
            pool = s["pool"].double()
            pool.view(-1, case["h_kv"], D).index_copy_(0, s["slots"], row)
            return pool
        scale = row.abs().amax(-1) / E4M3_MAX
        # nearest representable values: steps of 2^-3 of the binade, 2^-9 below the normal range
        v = row / scale[..., None]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        v = torch.round(v / step) * step
        k8 = s["k8"].double()
        k8.view(-1, case["h_kv"], D).index_copy_(0, s["slots"], v)
        ks = s["scale"].double()
        ks.view(case["h_kv"], -1).index_copy_(1, s["slots"], scale.t().contiguous())
        return k8, ks
    if op == "read":
        rows = (s["k8"] if case["fp8"] else s["pool"]).double().flatten(0, 1).index_select(0, s["slots"])
        if case["fp8"]:
            rows *= s["scale"].double().flatten(1).index_select(1, s["slots"]).t().unsqueeze(-1)
        return rows
    if op == "decode":
        out, lse = [], []
        h, g = case["h_kv"], case["h_q"] // case["h_kv"]
        lens = s["lens"].tolist()
        for i in range(case["batch"]):
            n = lens[i]
            used = s["table"][i, :-(-n // PAGE)].long()
            k = (s["k8"][used].double() if n else torch.zeros((1, PAGE, h, D), dtype=torch.float64, device="cuda"))
            k = k.flatten(0, 1)[:n] * (s["scale"][:, used].double().flatten(1)[:, :n].t()[..., None] if n else 1.0)
            x = torch.einsum("shgd,nhd->hgsn", s["q"][i].double().view(case["s_q"], h, g, D), k) / math.sqrt(D)
            if case["causal"]:
                ahead = torch.arange(n, device="cuda")[None, :] > n - case["s_q"] + torch.arange(case["s_q"], device="cuda")[:, None]
                x.masked_fill_(ahead, -math.inf)
            z = torch.logsumexp(x, -1) if n else torch.full(x.shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
            p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[..., None])
            out.append(torch.einsum("hgsn,nhd->shgd", p, k[..., :DV]).reshape(case["s_q"], case["h_q"], DV))
            lse.append(z.reshape(case["h_q"], case["s_q"]))
        return torch.stack(out), torch.stack(lse)
    # one sequence after another on the host
    target, draft = s["target"].double().cpu().numpy(), None if s["draft"] is None else s["draft"].double().cpu().numpy()
    tokens, u, un, num = (s[k].cpu().numpy() for k in ("tokens", "u", "u_new", "n"))
    counts, made = np.zeros(case["batch"], np.int32), np.full((case["batch"], case["drafts"] + 1), -1, np.int32)
    for i in range(case["batch"]):
        r = 0
        while r < num[i] and np.float64(u[i, r]) * (1.0 if draft is None else draft[i, r, tokens[i, r]]) < target[i, r, tokens[i, r]]:
            made[i, r] = tokens[i, r]
            r += 1
        w = target[i, r].copy()
        if r < num[i]:
            if draft is None:
                w[tokens[i, r]] = max(w[tokens[i, r]] - 1.0, 0.0)
            else:
                w = np.maximum(w - draft[i, r], 0.0)
            if not w.sum() > 0:
                w = target[i, r].copy()
        c = np.cumsum(w)
        j = int(np.searchsorted(c, np.float64(un[i]) * c[-1], side="right"))
        made[i, r] = j if j < case["vocab"] else int(np.nonzero(w)[0][-1])
        counts[i] = r
    return torch.from_numpy(counts), torch.from_numpy(made)
