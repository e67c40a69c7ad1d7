"""The operators around a decode layer's compressed projections: per-head norms
with the position rotation, appending to a paged cache, and attention over that
cache for a batch that shares prefixes.  Each as it is measured: its cases, its
inputs, its plain form in elementary torch operations, and its definition in
64 bits.

The fused q/k/v projection of a compressed matrix gives FP32 rows
[tokens, (heads + 2 kv_heads) x dim]; q, k and v are views of them.
"""
import math
import random

import torch

own = False

EPS = 1e-6
THETA = 500000.0


# ---- cases ------------------------------------------------------------------

def listed():
    """32 query heads over 8 key heads of 128 is the layout of the decode stacks
    that the benchmark runs (their q/k/v projections have 4096 + 2 x 1024 rows);
    64 rows is the most that one GEMV call takes."""
    return [
        # One token of one stream: what a chat pays per layer beside its GEMVs.
        dict(name="qk_token", op="qk", tokens=1, heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, norm=True, dtype="fp32", far=4000),
        # An odd batch of streams at far positions, a part of each head rotated in pairs.
        dict(name="qk_batch", op="qk", tokens=61, heads=28, kv_heads=4, dim=128, rotary=64,
             interleaved=True, norm=True, dtype="fp32", far=1000000),
        # A whole prompt, from 16-bit projections.
        dict(name="qk_prompt", op="qk", tokens=8192, heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, norm=True, dtype="bf16", far=131072),
        # One token of one stream into its pages.
        dict(name="append_token", op="append", batch=1, chunk=1, ragged=False, heads=32,
             kv_heads=8, dim=128, rotary=128, interleaved=False, norm=True, dtype="fp32",
             page=16, own_lo=700, own_hi=700, groups=0, prefix_lo=0, prefix_hi=0),
        # A full decode batch behind one system prompt.
        dict(name="append_batch", op="append", batch=64, chunk=1, ragged=False, heads=32,
             kv_heads=8, dim=128, rotary=128, interleaved=False, norm=True, dtype="fp32",
             page=16, own_lo=1, own_hi=500, groups=1, prefix_lo=4096, prefix_hi=4096),
        # Chunks of four prompts of unequal lengths, padded to the longest; no norms.
        dict(name="append_chunk", op="append", batch=4, chunk=1024, ragged=True, heads=32,
             kv_heads=8, dim=128, rotary=128, interleaved=False, norm=False, dtype="bf16",
             page=32, own_lo=1500, own_hi=2500, groups=0, prefix_lo=0, prefix_hi=0),
        # One token of one stream, a short context: latency.
        dict(name="attend_token", op="attend", batch=1, chunk=1, ragged=False, heads=32,
             kv_heads=8, dim=128, page=16, own_lo=1003, own_hi=1003, groups=0, prefix_lo=0,
             prefix_hi=0),
        # Eight streams a few tokens behind a short shared prompt.
        dict(name="attend_short", op="attend", batch=8, chunk=1, ragged=False, heads=32,
             kv_heads=8, dim=128, page=16, own_lo=1, own_hi=60, groups=1, prefix_lo=777,
             prefix_hi=777),
        # Four prompts with eight beams each, heads of 64.
        dict(name="attend_groups", op="attend", batch=32, chunk=1, ragged=False, heads=32,
             kv_heads=8, dim=64, page=32, own_lo=20, own_hi=250, groups=4, prefix_lo=2000,
             prefix_hi=4096),
        # A prompt's chunk of 64 rows against what is cached already.
        dict(name="attend_chunk", op="attend", batch=1, chunk=64, ragged=False, heads=32,
             kv_heads=8, dim=128, page=64, own_lo=16400, own_hi=16400, groups=0, prefix_lo=0,
             prefix_hi=0),
        # A full decode batch behind a shared prompt of 8k tokens.
        dict(name="attend_batch", op="attend", batch=64, chunk=1, ragged=False, heads=32,
             kv_heads=8, dim=128, page=16, own_lo=1, own_hi=500, groups=1, prefix_lo=8200,
             prefix_hi=8200),
        # A full decode batch behind a document of 32k tokens, long answers.
        dict(name="attend_document", op="attend", batch=64, chunk=1, ragged=False, heads=32,
             kv_heads=8, dim=128, page=16, own_lo=100, own_hi=1900, groups=1, prefix_lo=32768,
             prefix_hi=32768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "append", "attend", "attend"])
    heads, kv_heads = rng.choice([(32, 8), (28, 4), (16, 2), (8, 8), (24, 8), (10, 2), (16, 1)])
    if op == "qk":
        dim = rng.choice([64, 80, 96, 128, 256])
        return dict(op=op, tokens=_log(rng, 1, 4096), heads=heads, kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.7, dtype=rng.choice(["fp32", "bf16"]),
                    far=_log(rng, 100, 2000000))
    dim = rng.choice([64, 128])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    batch = _log(rng, 1, 64)
    groups = rng.choice([0, 1, 1, min(batch, 3)])
    if op == "append":
        chunk = rng.choice([1, 1, _log(rng, 2, 4096 // batch)])
        hi = chunk + _log(rng, 1, 1000)
        far = _log(rng, 1, 30000)
        return dict(op=op, batch=batch, chunk=chunk, ragged=chunk > 1 and rng.random() < 0.5,
                    heads=heads, kv_heads=kv_heads, dim=dim, rotary=dim,
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.5,
                    dtype=rng.choice(["fp32", "bf16"]), page=page,
                    own_lo=chunk + rng.randrange(hi - chunk), own_hi=hi, groups=groups,
                    prefix_lo=far // 2, prefix_hi=far)
    chunk = rng.choice([1, 1, 1, rng.randint(2, max(2, 64 // batch))])
    far = _log(rng, 1, 32768 // max(1, groups))
    hi = chunk + _log(rng, 1, min(34000 - far * (groups > 0), 60000 // batch))
    return dict(op=op, batch=batch, chunk=chunk, ragged=chunk > 1 and rng.random() < 0.5,
                heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                own_lo=chunk + rng.randrange(hi - chunk), own_hi=hi, groups=groups,
                prefix_lo=max(1, far // 2), prefix_hi=far)


def _lengths(case):
    """(own lengths, new tokens, prefix lengths, group starts) of a case: by the
    case alone, so that its work is known without its inputs."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    b, g = case["batch"], case["groups"]
    lens = [r.randint(case["own_lo"], case["own_hi"]) for _ in range(b)]
    new = [r.randint(1, case["chunk"]) if case["ragged"] else case["chunk"] for _ in range(b)]
    prefix = [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(g)]
    starts = [b * i // g for i in range(g + 1)] if g else []
    return lens, new, prefix, starts


def work(case):
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "qk":
        size = 4 if case["dtype"] == "fp32" else 2
        n = case["tokens"] * (h + hk) * d
        return {"bytes": n * (size + 2), "flops": n * 8}
    lens, new, prefix, starts = _lengths(case)
    if case["op"] == "append":
        size = 4 if case["dtype"] == "fp32" else 2
        n = sum(new) * (h + 2 * hk) * d
        return {"bytes": n * (size + 2), "flops": n * 8}
    rows = case["batch"] * case["chunk"]
    tokens = sum(lens) + sum(prefix)
    # Every real row meets its prefix and its own tokens up to itself.
    met = sum(n * (s - n) + n * (n + 1) // 2 for s, n in zip(lens, new))
    met += sum(sum(new[starts[i]:starts[i + 1]]) * p for i, p in enumerate(prefix))
    return {"bytes": 4 * tokens * hk * d + 4 * rows * h * d, "flops": 4 * met * h * d}


# ---- inputs -----------------------------------------------------------------

def _tables(counts, first, perm, device):
    """int32 [n, most] page tables: pages perm[first:...] dealt out in order, -1
    behind each row's last page; and the number of pages dealt."""
    most = max(1, max(counts))
    used = sum(counts)
    rows = torch.full((len(counts), most), -1, dtype=torch.int32, device=device)
    mask = torch.arange(most)[None, :] < torch.tensor(counts)[:, None]
    rows[mask.to(device)] = perm[first:first + used]
    return rows, used


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    s = {"case": case}

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if case["op"] != "attend":
        rows = case["tokens"] if case["op"] == "qk" else case["batch"] * case["chunk"]
        y = randn(rows, (h + 2 * hk) * d)
        y *= 0.5 + 2 * torch.rand((rows, 1), generator=gen, device=dev)
        s["y"] = y if case["dtype"] == "fp32" else y.bfloat16()
        s["freq"] = THETA ** (-torch.arange(case["rotary"] // 2, dtype=torch.float64,
                                            device=dev) * 2 / case["rotary"])
        s["qw"] = (1 + 0.2 * randn(d)).bfloat16() if case["norm"] else None
        s["kw"] = (1 + 0.2 * randn(d)).bfloat16() if case["norm"] else None
    if case["op"] == "qk":
        s["pos"] = torch.randint(0, case["far"], (case["tokens"],), generator=gen, device=dev)
        return s

    page = case["page"]
    lens, new, prefix, starts = _lengths(case)
    counts = [-(-n // page) for n in lens]
    shared = [-(-n // page) for n in prefix]
    total = sum(counts) + (sum(shared) if case["op"] == "attend" else 0)
    pool = total + max(1, total // 16)
    perm = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    s["k_pages"] = randn(pool, page, hk, d).bfloat16()
    s["v_pages"] = randn(pool, page, hk, d).bfloat16()
    s["table"], used = _tables(counts, 0, perm, dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["new"] = torch.tensor(new, dtype=torch.int32, device=dev) if case["ragged"] else None
    s["prefix_table"] = s["prefix_lens"] = s["starts"] = None
    if prefix:
        if case["op"] == "append":  # appending reads the prefixes' lengths, not their pages
            shared, perm, used = [1] * len(prefix), torch.zeros_like(perm).repeat(2), 0
        s["prefix_table"], _ = _tables(shared, used, perm, dev)
        s["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device=dev)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        if case["op"] == "append":
            s["prefix_table"] = s["prefix_table"].expand(-1, -(-max(prefix) // page)).contiguous()
        s["most"] = max(b - a for a, b in zip(starts, starts[1:]))
    if case["op"] == "attend":
        # Heads differ in how sharply they look; scores reach several units.
        q = randn(case["batch"] * case["chunk"], h, d)
        q *= 0.3 + 2.2 * torch.rand((1, h, 1), generator=gen, device=dev)
        s["q"] = q.bfloat16()
    return s


# ---- plain forms ------------------------------------------------------------

def _views(y, case):
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    q, k, v = y.split([h * d, hk * d, hk * d], dim=-1)
    return q.unflatten(-1, (h, d)), k.unflatten(-1, (hk, d)), v.unflatten(-1, (hk, d))


def _norm(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, pos, freq, interleaved):
    angle = pos.double()[:, None] * freq
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    n = freq.numel()
    r, rest = x[..., :2 * n], x[..., 2 * n:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        out = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = r[..., :n], r[..., n:]
        out = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((out, rest), -1)


def _places(s):
    """(sequence, own index, real) of every row [batch x chunk], and the prefix
    length of every sequence."""
    case = s["case"]
    b, t = case["batch"], case["chunk"]
    seq = torch.arange(b, device=s["lens"].device)
    i = torch.arange(t, device=seq.device)
    new = s["new"] if s["new"] is not None else torch.full_like(s["lens"], t)
    j = (s["lens"] - new)[:, None] + i
    real = (i < new[:, None]) & (j >= 0)
    base = torch.zeros_like(s["lens"])
    if s["starts"] is not None:
        inside = (seq[:, None] >= s["starts"][:-1]) & (seq[:, None] < s["starts"][1:])
        base = (inside * s["prefix_lens"]).sum(-1)
    return seq[:, None].expand(b, t), j, real, base


def _plain_qk(s):
    case = s["case"]
    q, k, _ = _views(s["y"], case)
    return [_rotate(_norm(x, w), s["pos"], s["freq"], case["interleaved"]).bfloat16()
            for x, w in ((q, s["qw"]), (k, s["kw"]))]


def _plain_append(s):
    case = s["case"]
    q, k, v = _views(s["y"], case)
    seq, j, real, base = _places(s)
    pos = (base[:, None] + j).flatten()
    q = _rotate(_norm(q, s["qw"]), pos, s["freq"], case["interleaved"])
    k = _rotate(_norm(k, s["kw"]), pos, s["freq"], case["interleaved"])
    on = real.flatten()
    q = torch.where(on[:, None, None], q, 0.0).bfloat16()
    at = j.flatten()[on]
    where = (s["table"][seq.flatten()[on], at // case["page"]].long(), at % case["page"])
    s["k_pages"][where] = k[on].bfloat16()
    s["v_pages"][where] = v[on].bfloat16()
    return [q, s["k_pages"], s["v_pages"]]


def _plain_attend(s):
    case = s["case"]
    b, t, h, hk, d = (case[x] for x in ("batch", "chunk", "heads", "kv_heads", "dim"))
    seq, j, real, _ = _places(s)
    q = s["q"].float().view(b, t, hk, h // hk, d) / math.sqrt(d)

    def tokens(pages, table):
        return pages[table.clamp(min=0).long()].flatten(1, 2).float()

    kt, vt = tokens(s["k_pages"], s["table"]), tokens(s["v_pages"], s["table"])
    score = torch.einsum("btkgd,blkd->btkgl", q, kt)
    seen = real[..., None] & (torch.arange(kt.shape[1], device=q.device) <= j[..., None])
    score = score.masked_fill(~seen[:, :, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["starts"] is None:
        p = torch.exp(score - top.clamp(min=-1e30))
        out = torch.einsum("btkgl,blkd->btkgd", p, vt) / p.sum(-1, keepdim=True)
        return torch.where(real[..., None, None, None], out, 0.0).bfloat16().reshape(b * t, h, d)
    # Members of each prefix, padded to the largest group.
    member = s["starts"][:-1, None] + torch.arange(s["most"], device=q.device)
    inside = member < s["starts"][1:, None]
    member = member.clamp(max=b - 1)
    kp, vp = tokens(s["k_pages"], s["prefix_table"]), tokens(s["v_pages"], s["prefix_table"])
    far = torch.einsum("gmtkhd,glkd->gmtkhl", q[member], kp)
    live = torch.arange(kp.shape[1], device=q.device) < s["prefix_lens"][:, None]
    far = far.masked_fill(~live[:, None, None, None, None], -math.inf)
    top = torch.maximum(far.amax(-1, keepdim=True)[inside], top)
    p = torch.exp(score - top)
    top_far = torch.zeros_like(far[..., :1])
    top_far[inside] = top
    pf = torch.exp(far - top_far)
    num = torch.einsum("btkgl,blkd->btkgd", p, vt)
    num = num + torch.einsum("gmtkhl,glkd->gmtkhd", pf, vp)[inside]
    den = p.sum(-1, keepdim=True) + pf.sum(-1, keepdim=True)[inside]
    out = torch.where(real[..., None, None, None], num / den, 0.0)
    return out.bfloat16().reshape(b * t, h, d)


# ---- one pass ---------------------------------------------------------------

def _handles(s):
    """The cache and the batch's tables as a serving loop holds them."""
    from lossless_bf16_weight_nwc_b200 import paged
    if "kv" not in s:
        s["kv"] = paged.PagedKV(s["k_pages"], s["v_pages"])
        s["batch"] = paged.PagedBatch(s["table"], s["lens"], q_lens=s["new"],
                                      prefix_table=s["prefix_table"],
                                      prefix_lens=s["prefix_lens"], group_start=s["starts"])
    return s["kv"], s["batch"]


def run(s):
    case = s["case"]
    if not own:
        return {"qk": _plain_qk, "append": _plain_append, "attend": _plain_attend}[case["op"]](s)
    if case["op"] == "qk":
        from lossless_bf16_weight_nwc_b200 import paged
        q, k, _ = _views(s["y"], case)
        return list(paged.qk_norm_rope(q, k, s["pos"], s["freq"], q_weight=s["qw"],
                                       k_weight=s["kw"], eps=EPS,
                                       interleaved=case["interleaved"]))
    kv, batch = _handles(s)
    if case["op"] == "append":
        q, k, v = _views(s["y"], case)
        q = kv.append(batch, k, v, q=q, freq=s["freq"], q_weight=s["qw"], k_weight=s["kw"],
                      eps=EPS, interleaved=case["interleaved"])
        return [q, s["k_pages"], s["v_pages"]]
    return kv.attend(batch, s["q"])


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_head(x, w, pos, freq, interleaved):
    """x [rows, heads, dim] normed and rotated as complex numbers."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    n = freq.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device).expand(len(pos), n),
                       torch.outer(pos.double(), freq))[:, None]
    y = x.clone()
    even, odd = ((slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved
                 else (slice(0, n), slice(n, 2 * n)))
    z = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * turn
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "qk":
        y = s["y"].view(case["tokens"], h + 2 * hk, d)
        return [_exact_head(y[:, a:b], w, s["pos"], s["freq"], case["interleaved"])
                for a, b, w in ((0, h, s["qw"]), (h, h + hk, s["kw"]))]
    lens, new, prefix, starts = _lengths(case)
    t, page = case["chunk"], case["page"]
    group = [next((g for g in range(len(prefix)) if starts[g] <= b < starts[g + 1]), None)
             for b in range(case["batch"])]
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    if case["op"] == "append":
        y = s["y"].view(-1, h + 2 * hk, d)
        q = torch.zeros(y.shape[0], h, d, dtype=torch.float64, device=y.device)
        for b, (length, n) in enumerate(zip(lens, new)):
            first = length - n
            at = torch.arange(first, length, device=y.device)
            pos = at + (prefix[group[b]] if group[b] is not None else 0)
            rows = y[b * t:b * t + n]
            q[b * t:b * t + n] = _exact_head(rows[:, :h], s["qw"], pos, s["freq"],
                                             case["interleaved"])
            pages = s["table"][b].long()[at // page]
            kp[pages, at % page] = _exact_head(rows[:, h:h + hk], s["kw"], pos, s["freq"],
                                               case["interleaved"])
            vp[pages, at % page] = rows[:, h + hk:].double()
        return [q, kp, vp]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b, (length, n) in enumerate(zip(lens, new)):
        mine = s["table"][b].long()[:-(-length // page)]
        k, v = kp[mine].reshape(-1, hk, d)[:length], vp[mine].reshape(-1, hk, d)[:length]
        before = length - n
        if group[b] is not None:
            many = prefix[group[b]]
            far = s["prefix_table"][group[b]].long()[:-(-many // page)]
            k = torch.cat((kp[far].reshape(-1, hk, d)[:many], k))
            v = torch.cat((vp[far].reshape(-1, hk, d)[:many], v))
            before += many
        for i in range(n):
            m = before + i + 1
            q = s["q"][b * t + i].double().view(hk, h // hk, d)
            p = torch.softmax(torch.matmul(q, k[:m].permute(1, 2, 0)) / math.sqrt(d), -1)
            out[b * t + i] = torch.matmul(p, v[:m].transpose(0, 1)).reshape(h, d)
    return out
