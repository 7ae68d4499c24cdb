"""Cases of the paged serving path: rotary positions, filling a paged key-value cache, one
new token's Infini-attention over it, and eviction from it by accumulated attention weight.

`run` computes each operator in elementary torch operations (32 bits, angles in 64), or,
where `own` is true, by the library's calls.  Head layouts are those of the workloads: 32
query heads on 8 key/value heads at d = 128, 16 on 16 at d = 128, 8 on 8 at d = 64, 2 on 2 at
d = 32.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the prefill of a grouped-head sequence: projections in token order, rotated into head order
        dict(name="rotary_prefill_gqa", op="rotary", B=1, H=32, Hkv=8, L=32768, d=128, rot=128,
             dtype="bf16", interleaved=False, tokenmajor=True, start=0, far=False),
        # a short batch, neighbouring pairs, half of the head rotated, positions given per token
        dict(name="rotary_short_partial", op="rotary", B=2, H=8, Hkv=8, L=1021, d=64, rot=32,
             dtype="bf16", interleaved=True, tokenmajor=True, start=0, far=True),
        # gradients of a long stream's last part, positions near a million
        dict(name="rotary_backward_far", op="rotary_bwd", B=1, H=16, Hkv=16, L=16383, d=128,
             rot=128, dtype="f32", interleaved=False, tokenmajor=False, start=1032193, far=False),
        # a ragged batch of prompts put into the pages
        dict(name="append_prompts", op="append", B=16, H=32, Hkv=8, T=2048, d=128, page=64,
             dtype="bf16", longest=2048, tokenmajor=True),
        # one token for each sequence of a large batch
        dict(name="append_token", op="append", B=64, H=32, Hkv=8, T=1, d=128, page=16,
             dtype="bf16", longest=2000, tokenmajor=True),
        # the smallest step: one short sequence, plain attention (latency)
        dict(name="decode_short", op="decode", B=1, H=8, Hkv=8, longest=64, d=64, page=16,
             dtype="bf16", memory=False, weights=False, rot=64, ragged=False),
        # a serving batch: ragged segments, memory and gate, weights kept for eviction
        dict(name="decode_batch_infini", op="decode", B=32, H=32, Hkv=8, longest=2047, d=128,
             page=64, dtype="bf16", memory=True, weights=True, rot=128, ragged=True),
        # one stream whose whole history is still in the cache
        dict(name="decode_long", op="decode", B=1, H=32, Hkv=8, longest=1000003, d=128, page=64,
             dtype="bf16", memory=True, weights=False, rot=128, ragged=False),
        # 32-bit activations, one query head for each key/value head
        dict(name="decode_f32", op="decode", B=6, H=8, Hkv=8, longest=5000, d=64, page=32,
             dtype="f32", memory=True, weights=True, rot=0, ragged=True),
        # a batch cut from two segments' rows to one, without memory
        dict(name="evict_batch", op="evict", B=16, H=32, Hkv=8, longest=4096, budget=2048,
             recent=512, d=128, page=64, dtype="bf16", memory=False, ragged=True),
        # a long prompt cut to one segment, the evicted rows folded into the memory
        dict(name="evict_prompt_fold", op="evict", B=1, H=32, Hkv=8, longest=65500, budget=2048,
             recent=256, d=128, page=64, dtype="bf16", memory=True, ragged=False),
        # the smallest cut
        dict(name="evict_small", op="evict", B=1, H=2, Hkv=2, longest=100, budget=64, recent=16,
             d=32, page=8, dtype="f32", memory=True, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_bwd", "append", "decode", "decode", "evict", "evict"])
    H, Hkv, d = rng.choice([(32, 8, 128), (16, 16, 128), (8, 8, 64), (2, 2, 32)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    row = Hkv * d * (2 if dtype == "bf16" else 4)
    if op in ("rotary", "rotary_bwd"):
        B = rng.choice([1, 1, 2, 3, 5])
        L = _log(rng, 1, min(65536, (1 << 27) // (B * (H + Hkv) * d)))
        return dict(op=op, B=B, H=H, Hkv=Hkv, L=L, d=d, rot=rng.choice([d, d, d // 2, d // 4 + 2]),
                    dtype=dtype, interleaved=rng.random() < 0.5, tokenmajor=rng.random() < 0.5,
                    start=rng.choice([0, rng.randrange(1 << 20)]), far=rng.random() < 0.3)
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "append":
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(8192, (1 << 27) // (B * row))))
        return dict(op=op, B=B, H=H, Hkv=Hkv, T=T, d=d, page=page, dtype=dtype,
                    longest=T + rng.randrange(1, 512), tokenmajor=rng.random() < 0.5)
    if op == "decode":
        B = _log(rng, 1, 96)
        n = _log(rng, 1, max(64, min(400000, (1 << 30) // (B * row))))
        return dict(op=op, B=B, H=H, Hkv=Hkv, longest=n, d=d, page=page, dtype=dtype,
                    memory=rng.random() < 0.6, weights=rng.random() < 0.5,
                    rot=rng.choice([0, d, d // 2]), ragged=B > 1 and rng.random() < 0.7)
    B = _log(rng, 1, 32)
    n = _log(rng, 40, max(100, min(60000, (1 << 29) // (B * row))))
    budget = rng.randrange(max(1, n // 16), n + 1)
    return dict(op=op, B=B, H=H, Hkv=Hkv, longest=n, budget=budget,
                recent=rng.randrange(0, budget + 1), d=d, page=page, dtype=dtype,
                memory=rng.random() < 0.5, ragged=B > 1 and rng.random() < 0.7)


def _freq(rot):
    return torch.pow(torch.tensor(10000.0, dtype=torch.float64),
                     -torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1)).cuda()


def _lens(c, cpu):
    """Rows in the cache of each sequence: one at least as long as the case says."""
    if not c.get("ragged", False):
        return torch.full((c["B"],), c["longest"], dtype=torch.int32)
    n = torch.randint(0, c["longest"] + 1, (c["B"],), generator=cpu, dtype=torch.int32)
    n[int(torch.randint(0, c["B"], (1,), generator=cpu))] = c["longest"]
    return n


def _tables(lists, cpu, width):
    """Page tables for several numbers of pages, no page used twice; unused entries -1."""
    P = sum(len(x) * w for x, w in zip(lists, width)) + 3
    perm, at, out = torch.randperm(P, generator=cpu).to(torch.int32), 0, []
    for x, w in zip(lists, width):
        t = torch.full((len(x), w), -1, dtype=torch.int32)
        for b, n in enumerate(x.tolist()):
            t[b, :n] = perm[at:at + n]
            at += n
        out.append(t.cuda())
    return P, out


def prepare(c, seed):
    gpu = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    cpu = torch.Generator().manual_seed(seed * 2 + 1)
    dt, B, Hkv, d = _DT[c["dtype"]], c["B"], c["Hkv"], c["d"]

    def normal(*shape, dtype=dt):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        return x.normal_(generator=gpu)

    def heads(n, rows):
        if c.get("tokenmajor", False):
            return normal(B, rows, n, d).transpose(1, 2)
        return normal(B, n, rows, d)

    s = dict(case=c)
    if c["op"] in ("rotary", "rotary_bwd"):
        s.update(q=heads(c["H"], c["L"]), k=heads(Hkv, c["L"]), freq=_freq(c["rot"]), positions=None)
        if c["far"]:   # packed documents: positions start again inside a row
            s["positions"] = torch.randint(0, 1 << 20, (B, 1), generator=cpu).cuda() + \
                torch.arange(c["L"], device="cuda").remainder(max(1, c["L"] // 3))[None]
        return s
    page = c["page"]
    if c["op"] == "append":
        counts = torch.randint(0, c["T"] + 1, (B,), generator=cpu, dtype=torch.int32)
        counts[0] = c["T"]
        lens = (torch.rand(B, generator=cpu) * (c["longest"] - c["T"] + 1)).to(torch.int32)
        need = (lens + counts + page - 1) // page
        P, (table,) = _tables([need], cpu, [-(-c["longest"] // page)])
        return dict(s, k=heads(Hkv, c["T"]), v=heads(Hkv, c["T"]), lens=lens.cuda(),
                    counts=counts.cuda(), table=table, k_pages=normal(P, Hkv, page, d),
                    v_pages=normal(P, Hkv, page, d),
                    weights=torch.rand((P, Hkv, page), device="cuda", generator=gpu))
    lens = _lens(c, cpu)
    s["lens"] = lens.cuda()
    if c["memory"]:
        s["M"] = 0.1 * torch.rand((B, Hkv, d, d), device="cuda", generator=gpu)
        s["z"] = 1 + torch.rand((B, Hkv, d), device="cuda", generator=gpu)
        s["beta"] = normal(c["H"], dtype=torch.float32)
    if c["op"] == "decode":
        P, (s["table"],) = _tables([lens // page + 1], cpu, [c["longest"] // page + 1])
        s.update(q=normal(B, c["H"], d), k=normal(B, Hkv, d), v=normal(B, Hkv, d),
                 freq=None, positions=None)
        if c["rot"]:   # after an eviction a token's position is beyond its row
            far = torch.randint(0, 1 << 19, (B,), generator=cpu)
            s.update(freq=_freq(c["rot"]), positions=(lens.to(torch.int64) + far).cuda())
    else:
        P, (s["table"], s["dst"]) = _tables(
            [(lens + page - 1) // page, (lens.clamp(max=c["budget"]) + page - 1) // page], cpu,
            [-(-c["longest"] // page), -(-c["budget"] // page)])
    s["k_pages"], s["v_pages"] = normal(P, Hkv, page, d), normal(P, Hkv, page, d)
    if c["op"] == "evict" or c["weights"]:
        # few rows hold most of the weight, and some were never looked at
        w = torch.rand((P, Hkv, page), device="cuda", generator=gpu)
        s["weights"] = torch.where(w < 0.05, 0.0, w.pow(6) * 8)
    return s


# ---- plain forms -----------------------------------------------------------------------

def _rotate(x, ang, interleaved, back=False):
    """x [..., d] in 32 bits by the angles [..., rot/2] in 64."""
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    sin = -sin if back else sin
    rot = 2 * ang.shape[-1]
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((ya, yb), -1).flatten(-2) if interleaved else torch.cat((ya, yb), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_rotary(s, back):
    c = s["case"]
    pos = s["positions"] if s["positions"] is not None else \
        c["start"] + torch.arange(c["L"], device="cuda")[None]
    ang = (pos.double()[..., None] * s["freq"])[:, None]
    return [_rotate(x, ang, c["interleaved"], back).to(x.dtype) for x in (s["q"], s["k"])]


def _places(table, rows, page):
    """Page and slot of rows [B, n] of each sequence."""
    return table.long().clamp(min=0).gather(1, rows // page), rows % page


def _dense(pages, table, n):
    """Rows 0..n-1 of every sequence, [B, Hkv, n, ...]."""
    B, page = table.shape[0], pages.shape[2]
    x = pages[table[:, :-(-n // page)].long().clamp(min=0)].transpose(1, 2)
    return x.reshape(B, x.shape[1], -1, *pages.shape[3:])[:, :, :n]


def _plain_append(s):
    t = torch.arange(s["case"]["T"], device="cuda")[None]
    b, t = (t < s["counts"][:, None]).nonzero(as_tuple=True)
    rows = s["lens"].long()[b] + t
    page = s["case"]["page"]
    pg, slot = s["table"].long()[b, rows // page], rows % page
    s["k_pages"][pg, :, slot] = s["k"][b, :, t]
    s["v_pages"][pg, :, slot] = s["v"][b, :, t]
    s["weights"][pg, :, slot] = 0.0


def _feature(x):
    return torch.where(x > 0, x + 1, torch.exp(torch.clamp(x, max=0)))


def _plain_decode(s):
    c = s["case"]
    B, H, Hkv, d, page, n = c["B"], c["H"], c["Hkv"], c["d"], c["page"], c["longest"] + 1
    q, k = s["q"].float(), s["k"]
    if s["freq"] is not None:
        ang = (s["positions"].double()[:, None] * s["freq"])[:, None]
        q, k = _rotate(q, ang, False), _rotate(k, ang, False).to(k.dtype)
    at = s["lens"].long()[:, None]
    pg, slot = _places(s["table"], at, page)
    s["k_pages"][pg[:, 0], :, slot[:, 0]] = k
    s["v_pages"][pg[:, 0], :, slot[:, 0]] = s["v"]
    K, V = _dense(s["k_pages"], s["table"], n).float(), _dense(s["v_pages"], s["table"], n).float()
    rows = torch.arange(n, device="cuda")[None].expand(B, n)
    seen = rows <= at
    x = (q.view(B, Hkv, -1, d) @ K.transpose(2, 3)) / math.sqrt(d)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    out = p @ V
    if c["memory"]:
        f = _feature(q.view(B, Hkv, -1, d))
        den = (f @ s["z"][..., None])
        amem = torch.where(den == 0, 0.0, (f @ s["M"]) / den)
        g = (1 / (1 + torch.exp(-s["beta"]))).view(Hkv, -1)[None, :, :, None]
        out = g * amem + (1 - g) * out
    if c["weights"]:
        s["weights"][pg[:, 0], :, slot[:, 0]] = 0.0
        pg, slot = _places(s["table"], rows, page)
        b, r = seen.nonzero(as_tuple=True)
        s["weights"][pg[b, r], :, slot[b, r]] += p.sum(2).permute(0, 2, 1)[b, r]
    return out.reshape(B, H, d).to(s["q"].dtype)


def _plain_evict(s):
    c = s["case"]
    B, Hkv, page, n, budget = c["B"], c["Hkv"], c["page"], c["longest"], c["budget"]
    lens = s["lens"].long()
    w = _dense(s["weights"], s["table"], n)
    rows = torch.arange(n, device="cuda")[None]
    valid = (rows < lens[:, None])[:, None].expand(B, Hkv, n)
    recent = (rows >= lens[:, None] - c["recent"])[:, None]
    key = torch.where(valid, torch.where(recent, math.inf, w), -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices
    keep = torch.zeros_like(valid).scatter(2, order[..., :budget], True) & valid
    lens_out = s["lens"].clamp(max=budget)
    # kept rows in their old order, -1 behind them
    kept = torch.where(keep, rows[:, None], n).sort(dim=-1).values[..., :budget]
    kept = torch.where(kept == n, -1, kept).to(torch.int32)
    K, V = _dense(s["k_pages"], s["table"], n), _dense(s["v_pages"], s["table"], n)
    if c["memory"]:
        f = torch.where((valid & ~keep)[..., None], _feature(K.float()), 0.0)
        s["M"] += f.transpose(2, 3) @ V.float()
        s["z"] += f.sum(2)
    at = kept.long().clamp(min=0)
    b, r = (torch.arange(budget, device="cuda")[None] < lens_out[:, None]).nonzero(as_tuple=True)
    pg, slot = s["dst"].long()[b, r // page], r % page
    for_rows = at[..., None].expand(-1, -1, -1, c["d"])
    s["k_pages"][pg, :, slot] = K.gather(2, for_rows).transpose(1, 2)[b, r]
    s["v_pages"][pg, :, slot] = V.gather(2, for_rows).transpose(1, 2)[b, r]
    s["weights"][pg, :, slot] = w.gather(2, at).transpose(1, 2)[b, r]
    return lens_out, kept


def run(s):
    c = s["case"]
    if own:
        from compressive_memory_long_b200 import binding
    if c["op"] in ("rotary", "rotary_bwd"):
        if own:
            call = binding.rotary if c["op"] == "rotary" else binding.rotary_backward
            return call(s["q"], s["k"], s["freq"], positions=s["positions"], start=c["start"],
                        interleaved=c["interleaved"])
        return _plain_rotary(s, c["op"] == "rotary_bwd")
    if c["op"] == "append":
        if own:
            binding.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                 counts=s["counts"], weights=s["weights"])
        else:
            _plain_append(s)
        return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], weights=s["weights"])
    if c["op"] == "decode":
        if own:
            out = binding.paged_decode_step(
                s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                beta=s.get("beta"), M=s.get("M"), z=s.get("z"), weights=s.get("weights"),
                freq=s["freq"], positions=s["positions"])
        else:
            out = _plain_decode(s)
        got = dict(out=out, k_pages=s["k_pages"], v_pages=s["v_pages"])
        if c["weights"]:
            got["weights"] = s["weights"]
        return got
    if own:
        lens, kept = binding.paged_evict(
            s["k_pages"], s["v_pages"], s["weights"], s["table"], s["lens"], s["dst"],
            budget=c["budget"], recent=c["recent"], M=s.get("M"), z=s.get("z"))
    else:
        lens, kept = _plain_evict(s)
    got = dict(lens=lens, kept=kept, k_pages=s["k_pages"], v_pages=s["v_pages"], weights=s["weights"])
    if c["memory"]:
        got.update(M=s["M"], z=s["z"])
    return got


def work(c):
    es = 2 if c["dtype"] == "bf16" else 4
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["op"] in ("rotary", "rotary_bwd"):
        n = B * (H + Hkv) * c["L"] * d
        pos = 8 * B * c["L"] if c["far"] else 0
        return {"bytes": 2 * n * es + pos, "flops": 3 * n * c["rot"] // d}
    if c["op"] == "append":
        rows = c["T"] + (B - 1) * c["T"] / 2          # the first sequence is full, the others half on average
        return {"bytes": int(rows * Hkv * (4 * d * es + 4)), "flops": 0}
    if c["op"] == "decode":
        n = (c["longest"] * (B + 1) / 2 if c["ragged"] else c["longest"] * B) + B
        mem = B * Hkv * (d * d + d) * 4 if c["memory"] else 0
        byt = n * Hkv * 2 * d * es + mem + (B * H * 2 + B * Hkv * 4) * d * es
        byt += n * Hkv * 8 if c["weights"] else 0
        return {"bytes": int(byt), "flops": int(4 * n * H * d + (2 * B * H * d * d if c["memory"] else 0))}
    if c["ragged"]:                                   # lengths even over 0..longest, one the longest
        over = c["budget"] / c["longest"]
        kept = c["budget"] + (B - 1) * c["budget"] * (1 - over / 2)
        rows = c["longest"] * (B + 1) / 2
    else:
        kept, rows = B * c["budget"], B * c["longest"]
    byt = Hkv * (rows * 4 + kept * (4 * d * es + 4 + 4))
    if c["memory"]:
        byt += Hkv * ((rows - kept) * 2 * d * es + B * 2 * (d * d + d) * 4)
    return {"bytes": int(byt), "flops": int(2 * Hkv * (rows - kept) * d * d) if c["memory"] else 0}


# ---- the definitions in 64 bits, one sequence at a time --------------------------------------

def _exact_rotate(x, pos, freq, interleaved, back=False):
    """x [heads, n, d] at positions [n], as products of complex numbers."""
    x, r = x.double(), freq.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       (-1.0 if back else 1.0) * pos.double()[:, None] * freq)
    y = x.clone()
    if interleaved:
        re, im = slice(0, 2 * r, 2), slice(1, 2 * r, 2)
    else:
        re, im = slice(0, r), slice(r, 2 * r)
    w = torch.complex(x[..., re], x[..., im]) * turn
    y[..., re], y[..., im] = w.real, w.imag
    return y


def _exact_feature(x):
    return torch.clamp(x, min=0) + torch.exp(-torch.clamp(-x, min=0))


def exact(c, seed):
    s = prepare(c, seed)
    B, Hkv = c["B"], c["Hkv"]
    if c["op"] in ("rotary", "rotary_bwd"):
        got = []
        for x in (s["q"], s["k"]):
            y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            for b in range(B):
                pos = s["positions"][b] if s["positions"] is not None else \
                    torch.arange(c["start"], c["start"] + c["L"], device="cuda")
                y[b] = _exact_rotate(x[b], pos, s["freq"], c["interleaved"], c["op"] == "rotary_bwd")
            got.append(y)
        return got
    page, Kp, Vp = c["page"], s["k_pages"].double(), s["v_pages"].double()
    W = s["weights"].double() if "weights" in s else None
    table = s["table"].tolist()
    lens = s["lens"].tolist()

    def places(tab, rows):
        """Page numbers and slots of the rows of one sequence."""
        r = torch.as_tensor(rows, device="cuda")
        return torch.tensor(tab, device="cuda")[r // page], r % page

    if c["op"] == "append":
        for b, m in enumerate(s["counts"].tolist()):
            if m:
                p, t = places(table[b], range(lens[b], lens[b] + m))
                Kp[p, :, t] = s["k"][b, :, :m].double().transpose(0, 1)
                Vp[p, :, t] = s["v"][b, :, :m].double().transpose(0, 1)
                W[p, :, t] = 0
        return dict(k_pages=Kp, v_pages=Vp, weights=W)
    if c["op"] == "decode":
        G = c["H"] // Hkv
        out = torch.empty((B, c["H"], c["d"]), dtype=torch.float64, device="cuda")
        for b in range(B):
            q, k = s["q"][b].double(), s["k"][b].double()
            if s["freq"] is not None:
                at = s["positions"][b:b + 1]
                q = _exact_rotate(q[:, None], at, s["freq"], False)[:, 0]
                # what the cache holds is the rotated key in the cache's type
                k = _exact_rotate(k[:, None], at, s["freq"], False)[:, 0].to(s["k"].dtype).double()
            p, t = places(table[b], range(lens[b] + 1))
            Kp[p[-1], :, t[-1]], Vp[p[-1], :, t[-1]] = k, s["v"][b].double()
            for h in range(Hkv):
                qs = q[h * G:(h + 1) * G]
                x = qs @ Kp[p, h, t].T * c["d"] ** -0.5
                x = torch.exp(x - torch.logsumexp(x, 1, True))
                o = x @ Vp[p, h, t]
                if c["memory"]:
                    f = _exact_feature(qs)
                    g = torch.sigmoid(s["beta"][h * G:(h + 1) * G].double())[:, None]
                    o = g * (f @ s["M"][b, h].double()) / (f @ s["z"][b, h].double())[:, None] + (1 - g) * o
                out[b, h * G:(h + 1) * G] = o
                if c["weights"]:
                    W[p[-1], h, t[-1]] = 0
                    W[p, h, t] += x.sum(0)
        got = dict(out=out, k_pages=Kp, v_pages=Vp)
        if c["weights"]:
            got["weights"] = W
        return got
    M, z = (s["M"].double(), s["z"].double()) if c["memory"] else (None, None)
    kept = torch.full((B, Hkv, c["budget"]), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        m = min(n, c["budget"])
        if not n:
            continue
        p, t = places(table[b], range(n))
        pd, td = places(s["dst"][b].tolist(), range(m))
        for h in range(Hkv):
            w = W[p, h, t].cpu().numpy()
            old = max(0, n - c["recent"])
            # by weight downwards, then by row
            by = (-w[:old]).argsort(kind="stable")[:m - (n - old)] if n > m else range(old)
            rows = sorted(int(i) for i in by) + list(range(old, n))
            kept[b, h, :m] = torch.tensor(rows, dtype=torch.int32)
            r = torch.tensor(rows, device="cuda")
            if c["memory"]:
                gone = torch.ones(n, dtype=torch.bool, device="cuda")
                gone[r] = False
                f = _exact_feature(Kp[p[gone], h, t[gone]])
                M[b, h] += f.T @ Vp[p[gone], h, t[gone]]
                z[b, h] += f.sum(0)
            for X in (Kp, Vp, W):
                X[pd, h, td] = X[p[r], h, t[r]]
    got = dict(lens=torch.tensor([min(n, c["budget"]) for n in lens], dtype=torch.int32), kept=kept,
               k_pages=Kp, v_pages=Vp, weights=W)
    if c["memory"]:
        got.update(M=M, z=z)
    return got
