"""What the operators on packed sequences cost: cases, inputs, plain forms and exact values.

Four kinds of case: ``rope`` (rotary positions with several axes), ``packed`` (attention over packed
sequences of different lengths), ``train`` (the same with its gradients) and ``chunk`` (chunks of new
tokens appended to a paged KV cache and attended over it).
"""
import math
import random

import torch

own = False  # True: the framework's entry points; False: elementary torch operations


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token each of 64 sequences of a multimodal model: the rotation of a decode step
        dict(name="rope_step", op="rope", tokens=64, Hq=32, Hkv=8, D=128, sections="16,24,24", interleave=False,
             ladder=False, half=True, inverse=False, fused=True, far=False),
        # a long video prompt: time, height and width positions, axes interleaved over the pairs
        dict(name="rope_video", op="rope", tokens=32768, Hq=32, Hkv=8, D=128, sections="24,20,20", interleave=True,
             ladder=False, half=True, inverse=False, fused=True, far=False),
        # gradients of an image encoder's rotation: two axes, each with its own frequencies
        dict(name="rope_image_grad", op="rope", tokens=5003, Hq=16, Hkv=16, D=64, sections="16,16", interleave=False,
             ladder=True, half=False, inverse=True, fused=False, far=False),
        # a handful of short prompts: latency
        dict(name="packed_short", op="packed", seqs=7, lo=1, hi=90, lens=11, Hq=8, Hkv=2, D=128, causal=True, window=0,
             fused=True),
        # an ordinary batch of prompts
        dict(name="packed_prompts", op="packed", seqs=24, lo=100, hi=2000, lens=12, Hq=32, Hkv=8, D=128, causal=True,
             window=0, fused=True),
        # a few long documents
        dict(name="packed_long", op="packed", seqs=3, lo=4000, hi=20000, lens=13, Hq=32, Hkv=8, D=128, causal=True,
             window=0, fused=False),
        # an encoder over images of different sizes: every patch sees every patch of its image
        dict(name="packed_images", op="packed", seqs=12, lo=200, hi=4000, lens=14, Hq=16, Hkv=16, D=64, causal=False,
             window=0, fused=True),
        # a training step on packed documents
        dict(name="train_documents", op="train", seqs=16, lo=50, hi=2048, lens=15, Hq=32, Hkv=8, D=128, causal=True,
             window=0, fused=True),
        # a training step with a sliding window, three query heads to a K/V head, short odd documents
        dict(name="train_window", op="train", seqs=9, lo=33, hi=1500, lens=16, Hq=12, Hkv=4, D=64, causal=True,
             window=256, fused=False),
        # a few short turns on a small cache: latency
        dict(name="chunk_small", op="chunk", seqs=4, lo=100, hi=2000, new_lo=1, new_hi=40, singles=1, lens=17, Hq=8,
             Hkv=2, D=128, window=0),
        # a serving batch: most sequences bring one token, a few bring a chunk of their prompt
        dict(name="chunk_mixed", op="chunk", seqs=64, lo=512, hi=16384, new_lo=256, new_hi=1024, singles=60, lens=18,
             Hq=32, Hkv=8, D=128, window=0),
        # the next chunk of one very long prompt
        dict(name="chunk_long", op="chunk", seqs=1, lo=100000, hi=100000, new_lo=2048, new_hi=2048, singles=0, lens=19,
             Hq=32, Hkv=8, D=128, window=0),
    ]


_HEADS = [(32, 8), (8, 2), (16, 16), (12, 4), (8, 1), (10, 2), (4, 4), (32, 4)]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges (no name), no larger than the largest listed one of its kind."""
    largest = {}
    for c in listed():
        w = work(c)
        f, b = largest.get(c["op"], (0, 0))
        largest[c["op"]] = (max(f, w["flops"]), max(b, w["bytes"]))
    while True:
        op = rng.choice(["rope", "packed", "packed", "train", "train", "chunk", "chunk"])
        Hq, Hkv = rng.choice(_HEADS)
        D = rng.choice([64, 128, 128])
        if op == "rope":
            half = rng.random() < 0.5
            axes = rng.choice([1, 2, 3, 3, 4])
            total = rng.choice([D // 2, D // 2, D // 4])
            cuts = sorted(rng.sample(range(1, total), axes - 1))
            sections = [b - a for a, b in zip([0] + cuts, cuts + [total])]
            interleave = False
            if axes > 1 and rng.random() < 0.5:
                interleave = True
                s = total // (axes + 1)
                sections = [total - s * (axes - 1)] + [s] * (axes - 1)
            c = dict(op=op, tokens=_log_int(rng, 1, 32768), Hq=Hq, Hkv=Hkv, D=D,
                     sections=",".join(str(x) for x in sections), interleave=interleave, ladder=rng.random() < 0.3,
                     half=half, inverse=rng.random() < 0.4, fused=rng.random() < 0.5, far=rng.random() < 0.3)
        elif op in ("packed", "train"):
            hi = _log_int(rng, 8, 20000 if op == "packed" else 2500)
            causal = rng.random() < 0.75
            c = dict(op=op, seqs=_log_int(rng, 1, 64), lo=max(1, hi // rng.choice([1, 3, 20, 1000])), hi=hi,
                     lens=rng.randrange(1 << 30), Hq=Hq, Hkv=Hkv, D=D, causal=causal,
                     window=_log_int(rng, 1, 2 * hi) if causal and rng.random() < 0.3 else 0,
                     fused=rng.random() < 0.5)
        else:
            hi = _log_int(rng, 1, 100000)
            seqs = _log_int(rng, 1, 64)
            new_hi = _log_int(rng, 1, 2048)
            c = dict(op=op, seqs=seqs, lo=max(1, hi // rng.choice([1, 4, 30])), hi=hi,
                     new_lo=max(1, new_hi // rng.choice([1, 4, 30])), new_hi=new_hi, singles=rng.randint(0, seqs),
                     lens=rng.randrange(1 << 30), Hq=Hq, Hkv=Hkv, D=D,
                     window=_log_int(rng, 1, 2 * hi) if rng.random() < 0.25 else 0)
        w = work(c)
        if w["flops"] <= largest[op][0] and w["bytes"] <= largest[op][1]:
            return c


def _lengths(case):
    """Sequence lengths of a packed batch, or (context, new tokens) of every sequence of a chunk batch."""
    rng = random.Random(case["lens"])
    if case["op"] != "chunk":
        return [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["seqs"])]
    ctx = [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["seqs"])]
    new = [1 if s < case["singles"] else _log_int(rng, case["new_lo"], case["new_hi"]) for s in range(case["seqs"])]
    order = list(range(case["seqs"]))
    rng.shuffle(order)
    return ctx, [new[i] for i in order]


def _pairs(n_new, n_keys, causal, window):
    """Visible (query, key) pairs of n_new queries at the end of n_keys keys."""
    if not causal:
        return n_new * n_keys
    first, last = n_keys - n_new + 1, n_keys  # keys visible to the first and the last query
    total = (first + last) * n_new // 2
    if window > 0:
        a = max(first, window + 1)  # queries that see more than the window
        if a <= last:
            total -= _sum_range(a - window, last - window)
    return total


def _sum_range(a, b):
    return (a + b) * (b - a + 1) // 2


def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rope":
        T, axes = case["tokens"], len(case["sections"].split(","))
        rot = sum(int(x) for x in case["sections"].split(","))
        return {"bytes": T * (Hq + Hkv) * D * 2 * 2 + 4 * axes * T, "flops": 6 * T * (Hq + Hkv) * rot}
    if case["op"] in ("packed", "train"):
        lens = _lengths(case)
        T = sum(lens)
        pairs = sum(_pairs(n, n, case["causal"], case["window"]) for n in lens) * Hq
        fwd = {"bytes": T * ((2 * Hq + 2 * Hkv) * D * 2 + Hq * 4), "flops": 4 * D * pairs}
        if case["op"] == "packed":
            return fwd
        return {"bytes": fwd["bytes"] + T * (2 * Hq + 2 * Hkv) * D * 2, "flops": 14 * D * pairs}
    ctx, new = _lengths(case)
    w = case["window"]
    pairs = sum(_pairs(n, c + n, True, w) for c, n in zip(ctx, new)) * Hq
    T = sum(new)
    keys = sum(min(c, w + n - 1) if w > 0 else c for c, n in zip(ctx, new))
    return {"bytes": (keys + 2 * T) * 2 * Hkv * D * 2 + T * Hq * (2 * D * 2 + 4), "flops": 4 * D * pairs}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _qkv(gen, T, Hq, Hkv, D, fused):
    """q, k, v [T, heads, D]: views of one projection's output, or tensors of their own."""
    if fused:
        x = _normal(gen, T, Hq + 2 * Hkv, D)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    return _normal(gen, T, Hq, D), _normal(gen, T, Hkv, D), _normal(gen, T, Hkv, D)


def _positions(case, seed):
    """[axes, T] positions of a prompt that alternates text runs and grids of patches."""
    rng = random.Random(seed)
    axes, T = len(case["sections"].split(",")), case["tokens"]
    cols, at = [], (rng.randrange(1 << 20, 1 << 24) if case["far"] else rng.randrange(0, 100))
    while len(cols) < T:
        if rng.random() < 0.5:
            n = rng.randint(1, 200)
            cols += [[at + i] * axes for i in range(n)]
            at += n
        else:
            h, w = rng.randint(2, 40), rng.randint(2, 40)
            for f in range(rng.randint(1, 4)):
                for i in range(h * w):
                    cols.append([at + x for x in (f, i // w, i % w, f)][:axes])
            at += max(h, w)
    return torch.tensor(cols[:T], dtype=torch.int32).t().contiguous().cuda()


def prepare(case, seed):
    g = _gen(seed)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    st = {"case": case}
    if case["op"] == "rope":
        st["q"], st["k"], _ = _qkv(g, case["tokens"], Hq, Hkv, D, case["fused"])
        st["positions"] = _positions(case, seed)
        return st
    if case["op"] in ("packed", "train"):
        lens = _lengths(case)
        st["lens"] = lens
        st["q"], st["k"], st["v"] = _qkv(g, sum(lens), Hq, Hkv, D, case["fused"])
        st["cu"] = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
        if case["op"] == "train":
            st["dout"] = _normal(g, sum(lens), Hq, D)
        return st
    ctx, new = _lengths(case)
    total = [c + n for c, n in zip(ctx, new)]
    pages = [(n + 15) // 16 for n in total]
    pool = sum(pages) + 3
    perm = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(ctx), max(pages)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = perm[at:at + n]
        at += n
    st["lens"], st["new"] = total, new
    st["table"] = table.cuda()
    st["table_host"] = table
    st["seq_lens"] = torch.tensor(total, dtype=torch.int32).cuda()
    st["cu"] = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    st["k_pages"] = _normal(g, pool, Hkv, 16, D)
    st["v_pages"] = _normal(g, pool, Hkv, 16, D)
    st["q"], st["k_new"], st["v_new"] = _qkv(g, sum(new), Hq, Hkv, D, False)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    if own:
        from exact_attention_161_b200 import api
        if case["op"] == "rope":
            return api.attn_rope_axes(st["q"], st["k"], st["positions"],
                                      [int(x) for x in case["sections"].split(",")],
                                      interleave_axes=case["interleave"], per_axis_freq=case["ladder"],
                                      rope_half_split=case["half"], rope_base=10000.0, inverse=case["inverse"])
        if case["op"] == "packed":
            return api.attn_packed_fwd(st["q"], st["k"], st["v"], st["cu"], causal=case["causal"],
                                       window=case["window"])
        if case["op"] == "train":
            o, lse = api.attn_packed_fwd(st["q"], st["k"], st["v"], st["cu"], causal=case["causal"],
                                         window=case["window"])
            dq, dk, dv = api.attn_packed_bwd(st["q"], st["k"], st["v"], o, lse, st["dout"], st["cu"],
                                             causal=case["causal"], window=case["window"])
            return o, lse, dq, dk, dv
        o, lse = api.attn_chunk_paged(st["q"], st["k_pages"], st["v_pages"], st["table"], st["seq_lens"], st["cu"],
                                      k_new=st["k_new"], v_new=st["v_new"], window=case["window"])
        return o, lse, st["k_pages"], st["v_pages"]
    return {"rope": _rope_plain, "packed": _packed_plain, "train": _packed_plain, "chunk": _chunk_plain}[case["op"]](st)


def _pair_axes(case):
    """Axis and theta exponent (theta = base^-e) of every rotated pair."""
    sec = [int(x) for x in case["sections"].split(",")]
    total, n = sum(sec), len(sec)
    if case["interleave"]:
        axis = [i % n if i % n > 0 and i < n * sec[i % n] else 0 for i in range(total)]
    else:
        axis = [a for a, s in enumerate(sec) for _ in range(s)]
    if not case["ladder"]:
        return axis, [i / total for i in range(total)]
    seen, expo = [0] * n, []
    for a in axis:
        expo.append(seen[a] / sec[a])
        seen[a] += 1
    return axis, expo


def _rope_plain(st):
    case = st["case"]
    axis, expo = _pair_axes(case)
    half = len(axis)
    theta = 10000.0 ** -torch.tensor(expo, dtype=torch.float64, device="cuda")
    angle = st["positions"][torch.tensor(axis, device="cuda")].double() * theta[:, None]  # [pairs, T]
    sign = -1.0 if case["inverse"] else 1.0
    cos, sin = angle.cos().float().t()[:, None], (sign * angle.sin()).float().t()[:, None]
    out = []
    for x in (st["q"], st["k"]):
        y = x.float()
        if case["half"]:
            a, b = y[..., :half], y[..., half:2 * half]
        else:
            a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        r0, r1 = a * cos - b * sin, a * sin + b * cos
        z = y.clone()
        if case["half"]:
            z[..., :half], z[..., half:2 * half] = r0, r1
        else:
            z[..., 0:2 * half:2], z[..., 1:2 * half:2] = r0, r1
        out.append(z.to(torch.bfloat16))
    return tuple(out)


def _visible(i, j, causal, window):
    """Truth values [len(i), len(j)]: key j is visible to the query at position i."""
    ok = torch.ones(i.numel(), j.numel(), dtype=torch.bool, device=i.device)
    if causal:
        ok &= j[None] <= i[:, None]
    if window > 0:
        ok &= j[None] > i[:, None] - window
    return ok


def _attend_plain(q, k, v, causal, window, dout=None):
    """q [n, Hq, D] at the end of k, v [m, Hkv, D] (one sequence), in 32 bits, a block of queries at a time.
    Returns o [n, Hq, D], lse [Hq, n] and, with dout, dq, dk, dv."""
    n, Hq, D = q.shape
    m, Hkv = k.shape[0], k.shape[1]
    G, scale = Hq // Hkv, D ** -0.5
    qf = q.float().view(n, Hkv, G, D).permute(1, 2, 0, 3)          # [Hkv, G, n, D]
    kf, vf = k.float().permute(1, 0, 2), v.float().permute(1, 0, 2)  # [Hkv, m, D]
    o = torch.empty(Hkv, G, n, D, device=q.device)
    lse = torch.empty(Hkv, G, n, device=q.device)
    if dout is not None:
        df = dout.float().view(n, Hkv, G, D).permute(1, 2, 0, 3)
        dq, dk, dv = torch.empty_like(o), torch.zeros_like(kf), torch.zeros_like(vf)
    step = max(1, min(n, (1 << 28) // (Hq * m)))
    for a in range(0, n, step):
        b = min(n, a + step)
        hi = m - n + b if causal else m
        lo = max(0, m - n + a - window + 1) if window > 0 else 0
        i = torch.arange(m - n + a, m - n + b, device=q.device)
        j = torch.arange(lo, hi, device=q.device)
        qs = qf[:, :, a:b].reshape(Hkv, G * (b - a), D)
        s = (qs @ kf[:, lo:hi].transpose(1, 2)).view(Hkv, G, b - a, hi - lo) * scale
        s = s.masked_fill(~_visible(i, j, causal, window), float("-inf"))
        top = s.amax(-1, keepdim=True)
        p = (s - top).exp()
        l = p.sum(-1, keepdim=True)
        p = (p / l).view(Hkv, G * (b - a), hi - lo)
        ob = p @ vf[:, lo:hi]
        o[:, :, a:b] = ob.view(Hkv, G, b - a, D)
        lse[:, :, a:b] = (top + l.log())[..., 0]
        if dout is not None:
            db = df[:, :, a:b].reshape(Hkv, G * (b - a), D)
            dv[:, lo:hi] += p.transpose(1, 2) @ db
            ds = p * (db @ vf[:, lo:hi].transpose(1, 2) - (db * ob).sum(-1, keepdim=True)) * scale
            dq[:, :, a:b] = (ds @ kf[:, lo:hi]).view(Hkv, G, b - a, D)
            dk[:, lo:hi] += ds.transpose(1, 2) @ qs
    back = lambda x: x.permute(2, 0, 1, 3).reshape(n, Hq, D)
    if dout is None:
        return back(o), lse.view(Hq, n)
    return back(o), lse.view(Hq, n), back(dq), dk.permute(1, 0, 2), dv.permute(1, 0, 2)


def _packed_plain(st):
    case = st["case"]
    train = case["op"] == "train"
    q, k, v = st["q"], st["k"], st["v"]
    T, Hq, D = q.shape
    out = [torch.empty(T, Hq, D, dtype=torch.bfloat16, device=q.device), torch.empty(Hq, T, device=q.device)]
    if train:
        out += [torch.empty(x.shape, dtype=torch.bfloat16, device=q.device) for x in (q, k, v)]
    a = 0
    for n in st["lens"]:
        r = slice(a, a + n)
        got = _attend_plain(q[r], k[r], v[r], case["causal"], case["window"], st["dout"][r] if train else None)
        for x, y in zip(out, got):
            if x.dim() == 2:
                x[:, r] = y
            else:
                x[r] = y.to(x.dtype)
        a += n
    return tuple(out)


def _chunk_plain(st):
    case = st["case"]
    q, kp, vp = st["q"], st["k_pages"], st["v_pages"]
    T, Hq, D = q.shape
    Hkv = kp.shape[1]
    o, lse = torch.empty_like(q), torch.empty(T, Hq, device=q.device)
    a = 0
    for s, (m, n) in enumerate(zip(st["lens"], st["new"])):
        r = slice(a, a + n)
        pages = st["table"][s, :(m + 15) // 16].long()
        pos = torch.arange(m - n, m, device=q.device)
        kp[pages[pos // 16], :, pos % 16] = st["k_new"][r]
        vp[pages[pos // 16], :, pos % 16] = st["v_new"][r]
        lo = max(0, m - n - case["window"] + 1) // 16 if case["window"] > 0 else 0  # first page any query sees
        k = kp[pages[lo:]].transpose(1, 2).reshape(-1, Hkv, D)[:m - 16 * lo]
        v = vp[pages[lo:]].transpose(1, 2).reshape(-1, Hkv, D)[:m - 16 * lo]
        ob, lb = _attend_plain(q[r], k, v, True, case["window"])
        o[r], lse[r] = ob.to(o.dtype), lb.t()
        a += n
    return o, lse, kp, vp


# ------------------------------------------------------------------ exact values
def exact(case, seed):
    """The outputs of run(prepare(case, seed)) in 64 bits, from the definitions."""
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _rope_exact(st)
    window, causal = case["window"], case.get("causal", True)
    if case["op"] == "chunk":
        return _chunk_exact(st, window)
    cols = {name: [] for name in ("o", "lse", "dq", "dk", "dv")}
    a = 0
    for n in st["lens"]:
        r = slice(a, a + n)
        one = _sequence_exact(st["q"][r], st["k"][r], st["v"][r], causal, window,
                              st["dout"][r] if case["op"] == "train" else None)
        for name, x in zip(cols, one):
            cols[name].append(x)
        a += n
    return tuple(torch.cat(x, dim=1 if name == "lse" else 0) for name, x in cols.items() if x)


def _rope_exact(st):
    """Every pair as a complex number times e^(i angle)."""
    case = st["case"]
    sec = [int(x) for x in case["sections"].split(",")]
    R2, A = sum(sec), len(sec)
    owner = torch.zeros(R2, dtype=torch.long)
    if case["interleave"]:
        for a in range(1, A):
            owner[a:A * sec[a]:A] = a
    else:
        owner = torch.repeat_interleave(torch.arange(A), torch.tensor(sec))
    if case["ladder"]:
        e = torch.zeros(R2, dtype=torch.float64)
        for a in range(A):
            mine = (owner == a).nonzero()[:, 0]
            e[mine] = torch.arange(len(mine), dtype=torch.float64) / sec[a]
    else:
        e = torch.arange(R2, dtype=torch.float64) / R2
    theta = torch.pow(torch.tensor(10000.0, dtype=torch.float64), -e).cuda()
    pos = st["positions"].double().t()[:, owner.cuda()]
    turn = torch.polar(torch.ones_like(pos), pos * theta)[:, None]
    if case["inverse"]:
        turn = turn.conj()
    out = []
    for x in (st["q"], st["k"]):
        y = x.double()
        lead = y[..., :2 * R2]
        z = torch.complex(lead[..., :R2].contiguous(), lead[..., R2:].contiguous()) if case["half"] else \
            torch.view_as_complex(lead.reshape(*y.shape[:-1], R2, 2))
        z = z * turn
        lead = torch.cat([z.real, z.imag], -1) if case["half"] else torch.view_as_real(z).flatten(-2)
        out.append(torch.cat([lead, y[..., 2 * R2:]], -1))
    return tuple(out)


def _sequence_exact(q, k, v, causal, window, dout):
    """One sequence, one query head at a time, with whole score rows (4,096 queries at once)."""
    n, Hq, D = q.shape
    m, Hkv = k.shape[0], k.shape[1]
    dev, f64 = q.device, torch.float64
    O, L = torch.empty(n, Hq, D, dtype=f64, device=dev), torch.empty(Hq, n, dtype=f64, device=dev)
    grads = [torch.zeros(x.shape, dtype=f64, device=dev) for x in (q, k, v)] if dout is not None else None
    key = torch.arange(m, device=dev)
    for h in range(Hq):
        c = h * Hkv // Hq
        K, V = k[:, c].double(), v[:, c].double()
        for a in range(0, n, 4096):
            Q = q[a:a + 4096, h].double()
            at = (m - n + a + torch.arange(len(Q), device=dev))[:, None]
            S = torch.mm(Q, K.t()).div_(math.sqrt(D))
            if causal:
                S[key > at] = -math.inf
            if window > 0:
                S[key <= at - window] = -math.inf
            lse = torch.logsumexp(S, 1)
            P = S.sub_(lse[:, None]).exp_()
            o = torch.mm(P, V)
            O[a:a + 4096, h], L[h, a:a + 4096] = o, lse
            if grads is not None:
                G = dout[a:a + 4096, h].double()
                grads[2][:, c] += torch.mm(P.t(), G)
                dS = P * (torch.mm(G, V.t()) - (G * o).sum(1, keepdim=True))
                grads[0][a:a + 4096, h] = torch.mm(dS, K) / math.sqrt(D)
                grads[1][:, c] += torch.mm(dS.t(), Q) / math.sqrt(D)
    return (O, L) if grads is None else (O, L, *grads)


def _chunk_exact(st, window):
    kp, vp = st["k_pages"], st["v_pages"]
    Hkv, D = kp.shape[1], kp.shape[3]
    O, L, a = [], [], 0
    for s, (m, n) in enumerate(zip(st["lens"], st["new"])):
        t = torch.arange(m)
        row = st["table_host"][s].long()[t // 16].cuda()
        slot = (t % 16).cuda()
        kp[row[m - n:], :, slot[m - n:]] = st["k_new"][a:a + n]
        vp[row[m - n:], :, slot[m - n:]] = st["v_new"][a:a + n]
        o, lse = _sequence_exact(st["q"][a:a + n], kp[row, :, slot], vp[row, :, slot], True, window, None)
        O.append(o)
        L.append(lse.t())
        a += n
    return torch.cat(O), torch.cat(L), kp, vp
