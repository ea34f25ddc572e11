"""Packed-prompt and paged-cache attention: the cases they are measured at, and their plain forms.

Five operators: the forward and the training step (forward and backward) of attention over packed sequences of
different lengths, attention of new tokens over a paged cache, the append of new keys and values to that cache with
their rotary positions, and rotary positions by themselves (their backward is the rotation by the negative angle).

A case is plain values. Lengths are texts: "300,77,1" are three sequences.
"""

import math

import torch

own = False

PAGED = ("paged", "append")


# --------------------------------------------------------------------------- cases

def ints(text):
    return [int(x) for x in str(text).split(",")]


def listed():
    return [
        # A prefill batch of short chat prompts, every head with its own keys, in one pack.
        dict(name="packed_fwd_short_d64", op="packed_fwd", lens="300,1,77,128,129,255,64,33,2,190,256,17,100,200,31,96,169",
             hq=16, hkv=16, d=64, causal=True),
        # A long-context prefill with grouped heads: one long prompt, some medium ones and a stub.
        dict(name="packed_fwd_gqa_d128", op="packed_fwd", lens="8192,4097,2500,1024,511,60", hq=32, hkv=8, d=128,
             causal=True),
        # Training of a bidirectional encoder on packed documents.
        dict(name="packed_train_full_d64", op="packed_train", lens="700,512,300,129,128,127,100,52", hq=16, hkv=16,
             d=64, causal=False),
        # A training step of a decoder with grouped heads on documents packed to 8192 tokens.
        dict(name="packed_train_gqa_d128", op="packed_train", lens="4096,2048,1000,777,271", hq=32, hkv=8, d=128,
             causal=True),
        # One user, one new token, a short cache: latency.
        dict(name="paged_one_d64", op="paged", new="1", lens="1000", page=16, hq=16, hkv=16, d=64, causal=True),
        # A decode step of a server: one new token for each of 32 sequences of different lengths.
        dict(name="paged_decode_gqa_d128", op="paged", new=",".join(["1"] * 32),
             lens=",".join(str(500 + (i * 5077) % 7692) for i in range(32)), page=64, hq=32, hkv=8, d=128, causal=True),
        # Verification of four drafted tokens over long caches, few sequences.
        dict(name="paged_draft_long_d128", op="paged", new="4,4,4,4", lens="32768,30001,32000,31007", page=128, hq=64,
             hkv=8, d=128, causal=True),
        # A mixed step of a server: chunks of long prompts beside single tokens of running sequences.
        dict(name="paged_chunk_mixed_d128", op="paged", new="512,512,256,33,1,1,1,1", page=16,
             lens="8192,2048,16000,33,4000,129,2500,1", hq=32, hkv=8, d=128, causal=True),
        # The append of a decode step.
        dict(name="append_decode_d128", op="append", new=",".join(["1"] * 32),
             lens=",".join(str(500 + (i * 5077) % 7692) for i in range(32)), page=64, hq=32, hkv=8, d=128,
             sections="64", interleaved=False),
        # The append of a prefill step with image positions (time, height, width).
        dict(name="append_chunks_d128", op="append", new="4096,2048,1500,548", lens="8192,2048,16000,600", page=16,
             hq=32, hkv=8, d=128, sections="16,24,24", interleaved=False),
        # Queries and keys of a few tokens, neighbouring pairs, backward direction.
        dict(name="rope_back_d64", op="rope", tokens=64, hq=16, hkv=16, d=64, sections="32", interleaved=True, inverse=True),
        # Queries and keys of a packed batch with three axes.
        dict(name="rope_axes_d128", op="rope", tokens=16384, hq=32, hkv=8, d=128, sections="16,24,24", interleaved=False,
             inverse=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8] if d == 128 else [1, 4, 8, 16])
    hq = hkv * rng.choice([r for r in (1, 2, 3, 4, 5, 8) if hkv * r <= 32])
    op = rng.choice(["packed_fwd", "packed_train", "packed_train", "paged", "paged", "paged", "append", "rope"])
    if op in ("packed_fwd", "packed_train"):
        total, most = (spread(200, 16384), 8192) if op == "packed_fwd" else (spread(200, 8192), 4096)
        lens = []
        # As many sequences as keep the padded scores of the plain form below those of the largest listed case.
        while total > 0 and len(lens) < 24 and (len(lens) + 1) * max(lens + [1]) ** 2 * hq <= 5 * most * most * 32:
            lens.append(min(total, spread(1, most)))
            total -= lens[-1]
        rng.shuffle(lens)
        return dict(op=op, lens=",".join(map(str, lens)), hq=hq, hkv=hkv, d=d, causal=rng.random() < 0.75)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    sections = rng.choice(["%d" % (d // 2), "%d,%d,%d" % (d // 8, 3 * d // 16, 3 * d // 16), "%d" % (d // 4)])
    kind = rng.choice(["decode", "draft", "chunk"])
    count = spread(1, 48) if kind == "decode" else spread(1, 8)
    new, lens = [], []
    for _ in range(count):
        n = 1 if kind == "decode" else rng.randint(1, 8) if kind == "draft" else spread(1, 512)
        new.append(n)
        lens.append(n + (0 if rng.random() < 0.1 else spread(1, 8192 if kind == "decode" else 12000)))
    if op == "paged":
        return dict(op=op, new=",".join(map(str, new)), lens=",".join(map(str, lens)), page=page, hq=hq, hkv=hkv, d=d,
                    causal=kind == "decode" or rng.random() < 0.9)
    if op == "append":
        return dict(op=op, new=",".join(map(str, new)), lens=",".join(map(str, lens)), page=page, hq=hq, hkv=hkv, d=d,
                    sections=sections, interleaved=rng.random() < 0.3)
    return dict(op=op, tokens=spread(1, 12000), hq=hq, hkv=hkv, d=d, sections=sections, interleaved=rng.random() < 0.3,
                inverse=rng.random() < 0.5)


# --------------------------------------------------------------------------- inputs

def starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def inverse_frequencies(pairs, base=10000.0):
    """Radians per position of each pair, in 64 bits: base^(-i / pairs)."""
    return torch.pow(torch.tensor(base, dtype=torch.float64), -torch.arange(pairs, dtype=torch.float64) / pairs)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    d, hq, hkv = case["d"], case["hq"], case["hkv"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    s = dict(case)
    new = [case["tokens"]] if case["op"] == "rope" else ints(case["new"] if case["op"] in PAGED else case["lens"])
    tokens = sum(new)
    s["cu"] = torch.tensor(starts(new), dtype=torch.int32, device="cuda")
    s["q"], s["k"], s["v"] = normal(tokens, hq, d), normal(tokens, hkv, d), normal(tokens, hkv, d)
    s["most"] = max(new)
    s["scale"] = d ** -0.5
    if case["op"] == "packed_train":
        s["dout"] = normal(tokens, hq, d)
    if case["op"] in PAGED:
        # A pool with some spare pages; the sequences' pages lie in it in no order.
        lens, page = ints(case["lens"]), case["page"]
        used = [-(-n // page) for n in lens]
        pool = sum(used) + 4
        order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros(len(lens), max(used), dtype=torch.int32, device="cuda")
        for b, at in enumerate(starts(used)[:-1]):
            table[b, :used[b]] = order[at:at + used[b]]
        s["table"], s["most_len"] = table, max(lens)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["k_pages"], s["v_pages"] = normal(pool, hkv, page, d), normal(pool, hkv, page, d)
    if case["op"] in ("append", "rope"):
        sections = ints(case["sections"])
        s["sections"] = sections
        s["inv_freq"] = inverse_frequencies(sum(sections)).cuda()
        if case["op"] == "append" and len(sections) == 1:
            # The place of each new token in its sequence.
            s["positions"] = torch.cat([torch.arange(n - m, n, dtype=torch.int32, device="cuda")
                                        for m, n in zip(new, ints(case["lens"]))])[None]
        else:
            s["positions"] = torch.randint(0, 100000, (len(sections), tokens), generator=gen, device="cuda",
                                           dtype=torch.int32)
    return s


# --------------------------------------------------------------------------- plain forms

def padded(x, cu, most):
    """[T, H, d] -> [S, H, most, d] in 32 bits, and which places hold a token. A sequence's last token fills the rest."""
    at = torch.arange(most, device=x.device)
    n = (cu[1:] - cu[:-1]).long()
    rows = cu[:-1].long()[:, None] + torch.minimum(at[None], (n[:, None] - 1).clamp(min=0))
    return x[rows.clamp(max=x.shape[0] - 1)].permute(0, 2, 1, 3).float(), at[None] < n[:, None]


def unpadded(x, there):
    """[S, H, most, ...] -> [T, H, ...], the places that hold a token in their order."""
    return x.transpose(1, 2)[there]


def softmax_parts(q, k, seen, scale):
    """The weights, their rows' logarithm of the sum, for q [S, H, r, n, d], k [S, H, 1, m, d], seen [S, 1, 1, n, m]."""
    s = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    return p, (top + total.log())[..., 0]


def heads_at_once(s, q, m):
    """KV heads whose scores (S * r * n * m values each) are held at a time: those of all do not fit for long prompts."""
    each = q.shape[0] * (q.shape[1] // s["hkv"]) * q.shape[2] * m
    return max(1, min(s["hkv"], (1 << 31) // max(1, each)))


def plain_attention(s, q, k, v, seen, dout=None):
    """o, lse (and dq, dk, dv with `dout`), padded; q, dout [S, Hq, n, d], k, v [S, Hkv, m, d], seen [S, n, m]."""
    r, scale = s["hq"] // s["hkv"], s["scale"]
    q, k, v = q.unflatten(1, (s["hkv"], r)), k[:, :, None], v[:, :, None]
    seen = seen[:, None, None]
    step = heads_at_once(s, q.flatten(1, 2), k.shape[3])
    out = []
    for h in range(0, s["hkv"], step):
        qh, kh, vh = q[:, h:h + step], k[:, h:h + step], v[:, h:h + step]
        p, lse = softmax_parts(qh, kh, seen, scale)
        o = p @ vh
        if dout is None:
            out.append((o.flatten(1, 2), lse.flatten(1, 2)))
            continue
        do = dout.unflatten(1, (s["hkv"], r))[:, h:h + step]
        dv = (p.transpose(-1, -2) @ do).sum(2)
        ds = (do @ vh.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
        dq = (ds @ kh).mul_(scale)
        dk = (ds.transpose(-1, -2) @ qh).sum(2).mul_(scale)
        out.append((o.flatten(1, 2), lse.flatten(1, 2), dq.flatten(1, 2), dk, dv))
    return [torch.cat(x, 1) for x in zip(*out)]


def plain_packed(s):
    q, there = padded(s["q"], s["cu"], s["most"])
    k, v = padded(s["k"], s["cu"], s["most"])[0], padded(s["v"], s["cu"], s["most"])[0]
    seen = (there[:, :, None] & there[:, None, :]) if not s["causal"] else \
        (there[:, :, None] & there[:, None, :]).tril_()
    if s["op"] == "packed_fwd":
        o, lse = plain_attention(s, q, k, v, seen)
        return {"o": unpadded(o, there).bfloat16(), "lse": unpadded(lse, there).t()}
    # Places without a token take no part in the sums over queries.
    dout = padded(s["dout"], s["cu"], s["most"])[0] * there[:, None, :, None]
    o, lse, dq, dk, dv = plain_attention(s, q, k, v, seen, dout)
    return {"o": unpadded(o, there).bfloat16(), "lse": unpadded(lse, there).t(),
            "dq": unpadded(dq, there).bfloat16(), "dk": unpadded(dk, there).bfloat16(),
            "dv": unpadded(dv, there).bfloat16()}


def plain_paged(s):
    q, there = padded(s["q"], s["cu"], s["most"])
    # [S, pages, Hkv, page, d] -> [S, Hkv, m, d]
    k, v = (p[s["table"].long()].transpose(1, 2).flatten(2, 3)[:, :, :s["most_len"]].float()
            for p in (s["k_pages"], s["v_pages"]))
    key, lens = torch.arange(k.shape[2], device=k.device), s["lens"].long()
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    at = (lens - n)[:, None] + torch.arange(s["most"], device=k.device)[None]
    seen = there[:, :, None] & (key[None, None] < lens[:, None, None])
    if s["causal"]:
        seen = seen & (key[None, None] <= at[:, :, None])
    o, lse = plain_attention(s, q, k, v, seen)
    return {"o": unpadded(o, there).bfloat16(), "lse": unpadded(lse, there).t()}


def turns(s):
    """cos and sin [T, 1, pairs]; each pair goes by the axis of its section, angles in 64 bits."""
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"), output_size=sum(s["sections"]))
    angle = s["positions"].double()[axis].t() * s["inv_freq"]
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def plain_rotation(x, cos, sin, interleaved):
    pairs = cos.shape[-1]
    y = x.float()
    a, b = (y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2]) if interleaved else (y[..., :pairs], y[..., pairs:2 * pairs])
    c, e = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((c, e), -1).flatten(-2) if interleaved else torch.cat((c, e), -1)
    return torch.cat((turned, y[..., 2 * pairs:]), -1).bfloat16()


def plain_rope(s):
    cos, sin = turns(s)
    sin = -sin if s["inverse"] else sin
    return {"q": plain_rotation(s["q"], cos, sin, s["interleaved"]), "k": plain_rotation(s["k"], cos, sin, s["interleaved"])}


def plain_append(s):
    cos, sin = turns(s)
    q, k = plain_rotation(s["q"], cos, sin, s["interleaved"]), plain_rotation(s["k"], cos, sin, s["interleaved"])
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=q.shape[0])
    at = torch.arange(q.shape[0], device="cuda") - s["cu"][:-1].long()[seq] + (s["lens"].long() - n)[seq]
    page, slot = s["table"][seq, at // s["page"]].long(), at % s["page"]
    s["k_pages"][page, :, slot] = k
    s["v_pages"][page, :, slot] = s["v"]
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


PLAIN = {"packed_fwd": plain_packed, "packed_train": plain_packed, "paged": plain_paged, "append": plain_append,
         "rope": plain_rope}


# --------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return CALLS[s["op"]](s)
    return PLAIN[s["op"]](s)


def call_packed_fwd(s):
    from exact_io_aware_56_b200 import fa

    o, lse = fa.attention_packed_forward(s["q"], s["k"], s["v"], s["cu"], s["causal"], s["scale"])
    return {"o": o, "lse": lse}


def call_packed_train(s):
    from exact_io_aware_56_b200 import fa

    o, lse, resid = fa.attention_packed_forward(s["q"], s["k"], s["v"], s["cu"], s["causal"], s["scale"], residual=True)
    dq, dk, dv = fa.attention_packed_backward(s["q"], s["k"], s["v"], o, s["dout"], lse, s["cu"], s["causal"],
                                              s["scale"], o_resid=resid)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def call_paged(s):
    from exact_io_aware_56_b200 import fa

    o, lse = fa.attention_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], s["most"],
                                s["causal"], s["scale"])
    return {"o": o, "lse": lse}


def call_append(s):
    from exact_io_aware_56_b200 import fa

    q = fa.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], q=s["q"],
                        positions=s["positions"], inv_freq=s["inv_freq"], sections=s["sections"],
                        interleaved=s["interleaved"])
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def call_rope(s):
    from exact_io_aware_56_b200 import fa

    q, k = fa.rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["sections"], interleaved=s["interleaved"],
                   inverse=s["inverse"])
    return {"q": q, "k": k}


CALLS = {"packed_fwd": call_packed_fwd, "packed_train": call_packed_train, "paged": call_paged, "append": call_append,
         "rope": call_rope}


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    op = case["op"]
    if op == "rope":
        t = case["tokens"]
        return {"bytes": 4 * t * (hq + hkv) * d + 4 * t * len(ints(case["sections"])),
                "flops": 6 * t * (hq + hkv) * sum(ints(case["sections"]))}
    if op == "append":
        t = sum(ints(case["new"]))
        return {"bytes": 4 * t * (hq + 2 * hkv) * d + 4 * t * len(ints(case["sections"])) + 4 * t,
                "flops": 6 * t * (hq + hkv) * sum(ints(case["sections"]))}
    if op == "paged":
        new, lens = ints(case["new"]), ints(case["lens"])
        t = sum(new)
        seen = sum(n * m - (n * (n - 1) // 2 if case["causal"] else 0) for n, m in zip(new, lens))
        return {"bytes": 4 * t * hq * d + 4 * t * hq + 4 * hkv * d * sum(lens), "flops": 4 * hq * d * seen}
    lens = ints(case["lens"])
    t = sum(lens)
    seen = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
    if op == "packed_fwd":
        return {"bytes": 4 * t * hq * d + 4 * t * hkv * d + 4 * t * hq, "flops": 4 * hq * d * seen}
    # q, dout read, o, dq written; k, v read, dk, dv written; lse written. Two products forward, five backward.
    return {"bytes": 8 * t * hq * d + 8 * t * hkv * d + 4 * t * hq, "flops": 14 * hq * d * seen}


# --------------------------------------------------------------------------- the definition in 64 bits

def exact_rows(q, k, v, first, causal, scale):
    """One sequence, one query head: o [n, d], lse [n], and the weights; query i sits at place first + i."""
    z = torch.einsum("id,jd->ij", q, k) * scale
    if causal:
        i = torch.arange(q.shape[0], device=q.device) + first
        z = torch.where(torch.arange(k.shape[0], device=q.device)[None] <= i[:, None], z, -math.inf)
    lse = torch.logsumexp(z, 1)
    w = torch.exp(z - lse[:, None])
    return w @ v, lse, w


def exact_rotation(x, s, sign):
    """Each pair turned by (place on its section's axis) * (its frequency)."""
    axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    y = x.double().clone()
    pairs = len(axis)
    for i, a in enumerate(axis):
        t = sign * s["positions"][a].double() * s["inv_freq"][i]
        at, bt = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + pairs)
        u, w = x[:, :, at].double(), x[:, :, bt].double()
        y[:, :, at] = u * t.cos()[:, None] - w * t.sin()[:, None]
        y[:, :, bt] = u * t.sin()[:, None] + w * t.cos()[:, None]
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op, r, scale = s["op"], s["hq"] // s["hkv"], s["scale"]
    if op == "rope":
        sign = -1.0 if s["inverse"] else 1.0
        return {"q": exact_rotation(s["q"], s, sign), "k": exact_rotation(s["k"], s, sign)}
    if op == "append":
        k, kp, vp = exact_rotation(s["k"], s, 1.0), s["k_pages"].double(), s["v_pages"].double()
        at = 0
        for b, (n, m) in enumerate(zip(ints(case["new"]), ints(case["lens"]))):
            for page in range((m - n) // s["page"], (m - 1) // s["page"] + 1):
                lo, hi = max(m - n, page * s["page"]), min(m, (page + 1) * s["page"])
                where, rows = int(s["table"][b, page]), slice(at + lo - (m - n), at + hi - (m - n))
                kp[where, :, lo - page * s["page"]:hi - page * s["page"]] = k[rows].transpose(0, 1)
                vp[where, :, lo - page * s["page"]:hi - page * s["page"]] = s["v"][rows].double().transpose(0, 1)
            at += n
        return {"q": exact_rotation(s["q"], s, 1.0), "k_pages": kp, "v_pages": vp}
    new = ints(case["new"] if op == "paged" else case["lens"])
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["hq"], s["q"].shape[0], dtype=torch.float64, device="cuda")
    grads = {x: torch.zeros(s[x[1:]].shape, dtype=torch.float64, device="cuda") for x in ("dq", "dk", "dv")}
    at = 0
    for b, n in enumerate(new):
        rows = slice(at, at + n)
        at += n
        for h in range(s["hq"]):
            if op == "paged":
                m = ints(case["lens"])[b]
                places = torch.arange(m, device="cuda")
                where = s["table"][b].long()[places // s["page"]]
                k, v = (s[x][where, h // r, places % s["page"]].double() for x in ("k_pages", "v_pages"))
            else:
                m = n
                k, v = s["k"][rows, h // r].double(), s["v"][rows, h // r].double()
            q = s["q"][rows, h].double()
            o[rows, h], lse[h, rows], w = exact_rows(q, k, v, m - n, s["causal"], scale)
            if op == "packed_train":
                g = s["dout"][rows, h].double()
                grads["dv"][rows, h // r] += w.T @ g
                dz = w * (g @ v.T - (g * o[rows, h]).sum(1, keepdim=True)) * scale
                grads["dq"][rows, h] = dz @ k
                grads["dk"][rows, h // r] += dz.T @ q
    return {"o": o, "lse": lse, **(grads if op == "packed_train" else {})}
