"""The operators between a layer's projections on the GPU, against plain 64-bit
forms (paged_reference.py derives the bounds): norms with the rotation, the
paged append, and attention over shared prefixes, alone and as a layer runs
them together."""
import math

import numpy as np
import pytest

import paged_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def paged():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_bf16_weight_nwc_b200 import build
    build.build()
    from lossless_bf16_weight_nwc_b200 import paged as module
    torch.cuda.set_device(0)
    return module


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ---- norms and rotation -----------------------------------------------------

QK = [  # tokens, heads, kv_heads, dim, rotary, interleaved, weights, in, out
    (1, 32, 8, 128, 128, False, "bf16", "f32", "bf16"),
    (1, 1, 1, 8, 8, False, None, "bf16", "bf16"),
    (3, 5, 1, 64, 64, True, "f32", "bf16", "bf16"),
    (2, 3, 2, 80, 40, False, "bf16", "f32", "f32"),
    (65, 28, 4, 96, 96, True, "bf16", "f32", "bf16"),
    (7, 2, 2, 256, 256, False, "f32", "bf16", "f32"),
    (33, 9, 3, 256, 64, True, None, "f32", "bf16"),
    (5, 4, 4, 104, 48, False, "bf16", "bf16", "bf16"),
    (17, 8, 2, 128, 0, False, "bf16", "f32", "bf16"),
    (701, 32, 8, 128, 128, False, "bf16", "bf16", "bf16"),
    (2050, 10, 2, 64, 32, True, "f32", "f32", "bf16"),
    (1500, 24, 8, 256, 256, False, None, "f32", "f32"),
]
DT = {"bf16": torch.bfloat16, "f32": torch.float32} if torch else {}


def weights(g, kind, dim):
    return None if kind is None else (1 + 0.3 * randn(g, dim)).to(DT[kind])


@pytest.mark.parametrize("tokens,h,hk,dim,rotary,inter,wkind,tin,tout", QK)
def test_qk_norm_rope(paged, tokens, h, hk, dim, rotary, inter, wkind, tin, tout):
    g = gen(tokens + dim)
    y = (3 * randn(g, tokens, (h + 2 * hk) * dim)).to(DT[tin])
    q, k = y[:, :h * dim].unflatten(1, (h, dim)), y[:, h * dim:-hk * dim].unflatten(1, (hk, dim))
    pos = torch.randint(0, 200000, (tokens,), generator=g, device="cuda",
                        dtype=torch.int64 if tokens % 2 else torch.int32)
    freq = paged.rope_frequencies(rotary, 1e4) if rotary else None
    qw, kw = weights(g, wkind, dim), weights(g, wkind, dim)
    out = [torch.full(t.shape, math.nan, dtype=DT[tout], device="cuda") for t in (q, k)]
    before = y.clone()
    a, b = paged.qk_norm_rope(q, k, pos, freq, qw, kw, eps=1e-5, interleaved=inter, out=out)
    assert a is out[0] and b is out[1]
    for got, x, w in ((a, q, qw), (b, k, kw)):
        want, bound = ref.norm_rotate(x, w, pos, freq, inter, 1e-5)
        assert ref.close(got, want, bound, DT[tout])
    assert torch.equal(y, before)


LARGE = [  # as QK: enough tokens to fill the device, odd numbers of them
    (1301, 32, 8, 128, 128, False, "bf16", "bf16", "bf16"),
    (1301, 32, 8, 128, 128, True, "f32", "f32", "bf16"),
    (1203, 28, 4, 128, 128, False, None, "f32", "f32"),
    (1302, 12, 4, 64, 64, False, "bf16", "f32", "bf16"),
    (1303, 8, 8, 64, 64, True, "bf16", "bf16", "bf16"),
    (1299, 4, 4, 64, 64, True, None, "bf16", "f32"),
    (1201, 3, 1, 256, 256, True, "f32", "bf16", "bf16"),
    (1301, 7, 3, 128, 128, False, "bf16", "bf16", "bf16"),
    (1305, 6, 2, 96, 96, False, "bf16", "bf16", "bf16"),
    (1205, 32, 8, 128, 64, False, "bf16", "f32", "bf16"),
    (1205, 32, 8, 128, 0, False, "bf16", "bf16", "bf16"),
]


@pytest.mark.parametrize("tokens,h,hk,dim,rotary,inter,wkind,tin,tout", LARGE)
@pytest.mark.parametrize("form", ["both", "q", "k", "unaligned", "in place"])
def test_qk_norm_rope_of_prompts(paged, tokens, h, hk, dim, rotary, inter, wkind, tin, tout, form):
    """The forms that take several tokens a block: of whole heads and general, aligned
    and not, with q or k alone and in place."""
    g = gen(tokens + dim + rotary)
    off = 1 if form == "unaligned" else 0
    y = (2 * randn(g, tokens, (h + 2 * hk) * dim + off)).to(DT[tin])[:, off:]
    q, k, _ = (t.unflatten(1, (-1, dim)) for t in y.split([h * dim, hk * dim, hk * dim], 1))
    pos = torch.randint(0, 200000, (tokens,), generator=g, device="cuda")
    freq = paged.rope_frequencies(rotary, 1e4) if rotary else None
    qw, kw = weights(g, wkind, dim), weights(g, wkind, dim)
    want = [ref.norm_rotate(x, w, pos, freq, inter, 1e-6) for x, w in ((q, qw), (k, kw))]
    if form == "in place":
        out, tout = (q, k), tin
        v0 = y[:, -hk * dim:].clone()
    else:
        out = [torch.full(t.shape, math.nan, dtype=DT[tout], device="cuda") for t in (q, k)]
        y0 = y.clone()
    give = {"q": (q, None), "k": (None, k)}.get(form, (q, k))
    paged.qk_norm_rope(*give, pos, freq, qw, kw, interleaved=inter,
                       out=tuple(o if x is not None else None for o, x in zip(out, give)))
    for x, got, (w, bound) in zip(give, out, want):
        assert x is None and torch.isnan(got).all() or ref.close(got, w, bound, DT[tout])
    assert torch.equal(y[:, -hk * dim:], v0) if form == "in place" else torch.equal(y, y0)


def test_qk_far_and_negative_positions(paged):
    g = gen(1)
    pos = torch.tensor([0, -1, -5000, 2 ** 31 - 1, 2 ** 40 + 3, 10 ** 6], device="cuda")
    q = randn(g, 6, 4, 128)
    freq = paged.rope_frequencies(128, 5e5)
    a, none = paged.qk_norm_rope(q, None, pos, freq)
    assert none is None and a.dtype == torch.bfloat16
    want, bound = ref.norm_rotate(q, None, pos, freq, False, 0)
    # The definition's own angle is known to 2^-53 of 2^40 turns.
    assert ref.close(a, want, bound + 2.0 ** -12 * q.abs().amax(), torch.bfloat16)
    assert ref.close(a[[0, 1, 2, 5]], want[[0, 1, 2, 5]], bound[[0, 1, 2, 5]], torch.bfloat16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_qk_strides_alignment_and_in_place(paged, dtype):
    g = gen(2)
    freq = paged.rope_frequencies(64, 1e4)
    pos = torch.arange(9, device="cuda")
    # Odd row length, odd start, heads before tokens, a broadcast token.
    base = randn(g, 9, 4 * 64 + 1).to(DT[dtype])
    odd = base[:, 1:].unflatten(1, (4, 64))
    flat = randn(g, 4 * 9 * 64 + 3).to(DT[dtype])[3:].view(4, 9, 64).transpose(0, 1)
    wide = randn(g, 1, 4, 64).to(DT[dtype]).expand(9, 4, 64)
    for q in (odd, flat, wide):
        want, bound = ref.norm_rotate(q, None, pos, freq, False, 0)
        got, _ = paged.qk_norm_rope(q, None, pos, freq)
        assert ref.close(got, want, bound, torch.bfloat16)
        store = torch.zeros(9 * 4 * 65 + 1, dtype=DT[dtype], device="cuda")
        out = store[1:].view(9, 4, 65)[..., :64]
        paged.qk_norm_rope(q, None, pos, freq, out=(out, None))
        assert ref.close(out, want, bound, DT[dtype])
        assert not store[1:].view(9, 4, 65)[..., 64].any()
    want, bound = ref.norm_rotate(odd, None, pos, freq, False, 0)
    paged.qk_norm_rope(odd, None, pos, freq, out=(odd, None))      # in place
    assert ref.close(odd, want, bound, DT[dtype])


def test_qk_empty_and_special_values(paged):
    freq = paged.rope_frequencies(64, 1e4)
    q = torch.zeros((0, 4, 64), dtype=torch.float32, device="cuda")
    a, b = paged.qk_norm_rope(q, q, torch.zeros(0, dtype=torch.int32, device="cuda"), freq)
    assert a.shape == (0, 4, 64) and b.dtype == torch.bfloat16
    g = gen(3)
    x = randn(g, 3, 2, 64)
    x[0, 0, 5], x[1, 1, 7], x[2, 0] = math.nan, math.inf, 0.0
    w = torch.ones(64, device="cuda")
    a, _ = paged.qk_norm_rope(x, None, ints([4, 5, 6]), freq, w)
    good = torch.ones(3, 2, dtype=torch.bool)
    good[0, 0] = good[1, 1] = False
    want, bound = ref.norm_rotate(x, w, ints([4, 5, 6]), freq, False, 1e-6)
    assert torch.isnan(a[0, 0]).all() and not a[2, 0].any()
    assert torch.isnan(a[1, 1, 7]) and ref.close(a[good], want[good], bound[good], torch.bfloat16)


# ---- cache helpers ----------------------------------------------------------

class Case:
    """A cache with stale NaN behind every sequence's and prefix's last token."""

    def __init__(self, paged, seed, lens, kv_heads=2, dim=64, page=16, prefix=None, starts=None,
                 q_lens=None, heads_first=False, extra=2, poison=True, width=None):
        self.g = g = gen(seed)
        self.lens, self.q_lens, self.prefix, self.starts = lens, q_lens, prefix, starts
        count = [-(-max(n, 0) // page) for n in lens + (prefix or [])]
        pool = sum(count) + extra
        shape = (pool, kv_heads, page, dim) if heads_first else (pool, page, kv_heads, dim)
        k, v = randn(g, *shape).bfloat16(), randn(g, *shape).bfloat16()
        if heads_first:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        self.k, self.v = k, v
        perm = torch.randperm(pool, generator=g, device="cuda").int()
        width = width or max(count + [1]) + 1
        tables = torch.full((len(count), width), 2 ** 30, dtype=torch.int32, device="cuda")
        at = 0
        used = torch.zeros(pool, dtype=torch.bool, device="cuda")
        for i, c in enumerate(count):
            tables[i, :c] = perm[at:at + c]
            used[perm[at:at + c].long()] = True
            n = max((lens + (prefix or []))[i], 0)
            if poison and n % page:
                k[perm[at + c - 1], n % page:] = math.nan
                v[perm[at + c - 1], n % page:] = math.inf
            at += c
        if poison:
            k[~used], v[~used] = math.nan, math.nan
        n = len(lens)
        self.table, self.far = tables[:n], tables[n:] if prefix else None
        self.kv = paged.PagedKV(k, v)
        self.batch = paged.PagedBatch(
            self.table, ints(lens), None if q_lens is None else ints(q_lens), self.far,
            ints(prefix) if prefix else None, ints(starts) if prefix else None)

    def want(self, q, scale):
        return ref.attention(q, self.k, self.v, self.table, self.lens, self.q_lens, self.far,
                             self.prefix, self.starts, scale)

    def check(self, q, got, lse=None, scale=None):
        scale = scale if scale is not None else 1 / math.sqrt(q.shape[-1])
        want, bound, want_lse, lse_bound = self.want(q, scale)
        assert ref.close(got, want, bound, torch.bfloat16)
        if lse is not None:
            empty = want_lse == -math.inf
            assert torch.equal(lse == -math.inf, empty)
            off = (lse.double() - want_lse).abs()[~empty]
            assert bool((off <= lse_bound[~empty]).all())
        assert self.kv.device_error() == (0, 0)


def bits(t):
    return t.contiguous().view(torch.int16).clone()


# ---- append -----------------------------------------------------------------

APPEND = [  # lens, chunk, q_lens, kw
    ([1], 1, None, {}),
    ([700], 1, None, dict(kv_heads=8, dim=128)),
    ([5, 16, 17, 33], 1, None, dict(page=8)),
    ([40, 23, 64], 20, [20, 3, 0], dict(page=32, dim=80)),
    ([3, 300, 12, 9, 1], 1, None, dict(prefix=[100, 7], starts=[1, 3, 4])),
    ([66, 70], 66, [2, 66], dict(prefix=[1000], starts=[0, 2], heads_first=True, dim=128)),
    ([2, 0, 5, 1], 3, [2, 0, 3, 1], dict(prefix=[0, 31, 5], starts=[0, 1, 1, 4], page=16)),
    ([900, 1500], 700, [650, 700], dict(kv_heads=4, dim=256, page=128)),
    ([1] * 64, 1, None, dict(prefix=[4096] * 40, starts=list(range(41)), kv_heads=1)),
]


@pytest.mark.parametrize("lens,chunk,q_lens,kw", APPEND)
@pytest.mark.parametrize("tin,inter", [("f32", False), ("bf16", True)])
def test_append(paged, lens, chunk, q_lens, kw, tin, inter):
    c = Case(paged, len(lens) + chunk, lens, q_lens=q_lens, poison=False, **kw)
    hk, dim = c.kv.kv_heads, c.kv.dim
    h, rows = 3 * hk, len(lens) * chunk
    y = randn(c.g, rows, (h + 2 * hk) * dim).to(DT[tin])
    q, k, v = (t.unflatten(1, (-1, dim)) for t in y.split([h * dim, hk * dim, hk * dim], 1))
    freq, kw_ = paged.rope_frequencies(dim // 2 // 8 * 8, 1e4), weights(c.g, "bf16", dim)
    k0, v0 = c.k.clone(), c.v.clone()
    got = c.kv.append(c.batch, k, v, q=q, freq=freq, q_weight=kw_, k_weight=kw_, interleaved=inter)
    group = ref.groups_of(len(lens), c.starts)
    pos, real, where = [], [], []
    for b, n in enumerate(lens):
        fresh = chunk if q_lens is None else q_lens[b]
        base = c.prefix[group[b]] if group[b] is not None else 0
        for i in range(chunk):
            j = n - fresh + i
            pos.append(base + j)
            real.append(i < fresh)
            if real[-1]:
                where.append((b * chunk + i, int(c.table[b, j // c.kv.page_size]),
                              j % c.kv.page_size))
    pos, real = torch.tensor(pos, device="cuda"), torch.tensor(real, device="cuda")
    want, bound = ref.norm_rotate(q, kw_, pos, freq, inter, 1e-6)
    assert ref.close(got[real], want[real], bound[real], torch.bfloat16) and not got[~real].any()
    want, bound = ref.norm_rotate(k, kw_, pos, freq, inter, 1e-6)
    r, p, s = (torch.tensor(x, device="cuda") for x in zip(*where))
    assert ref.close(c.k[p, s], want[r], bound[r], torch.bfloat16)
    assert torch.equal(c.v[p, s], v[r].bfloat16())
    c.k[p, s], c.v[p, s] = k0[p, s], v0[p, s]
    assert torch.equal(bits(c.k), bits(k0)) and torch.equal(bits(c.v), bits(v0))
    assert c.kv.device_error() == (0, 0)


def test_tables_of_no_width(paged):
    """A prefix table without columns, for prefixes of no tokens; own tables without."""
    c = Case(paged, 17, [9, 30], poison=False)
    far = torch.zeros((1, 0), dtype=torch.int32, device="cuda")
    batch = paged.PagedBatch(c.table, ints(c.lens), None, far, ints([0]), ints([0, 2]))
    q, k, v = (randn(c.g, 2, n, 64).bfloat16() for n in (4, 2, 2))
    c.kv.append(batch, k, v)
    assert torch.equal(c.v[c.table[0, 0], 8], v[0])
    got, lse = c.kv.attend(batch, q, return_lse=True)
    c.check(q, got, lse)
    none = paged.PagedBatch(far.expand(2, 0), ints([0, 0]))
    assert not c.kv.attend(none, q).any() and c.kv.device_error() == (0, 0)
    k0 = c.k.clone()
    c.kv.append(paged.PagedBatch(far.expand(2, 0), ints([1, 1])), k, v)
    assert torch.equal(bits(c.k), bits(k0)) and c.kv.device_error() == (1, 4)


def test_empty_batches(paged):
    c = Case(paged, 18, [9], poison=False)
    table = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    none = paged.PagedBatch(table, ints([]))
    q, k = (torch.zeros((0, n, 64), dtype=torch.bfloat16, device="cuda") for n in (4, 2))
    assert c.kv.append(none, k, k, q=q).shape == (0, 4, 64)
    o, lse = c.kv.attend(none, q, return_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_append_large_batches_and_heads(paged):
    """More tokens than fill the device, heads that do not fill a warp's group."""
    for seqs, h, hk, dim in ((1500, 5, 1, 64), (1300, 3, 3, 80), (1250, 2, 1, 256)):
        c = Case(paged, seqs, [1 + i % 20 for i in range(seqs)], kv_heads=hk, dim=dim,
                 poison=False)
        y = randn(c.g, seqs, h + 2 * hk, dim).bfloat16()
        q, k, v = y.split([h, hk, hk], 1)
        freq = paged.rope_frequencies(dim // 16 * 16, 1e4)
        got = c.kv.append(c.batch, k, v, q=q, freq=freq)
        pos = torch.tensor(c.lens, device="cuda") - 1
        want, bound = ref.norm_rotate(q, None, pos, freq, False, 0)
        assert ref.close(got, want, bound, torch.bfloat16)
        at = (c.table[torch.arange(seqs, device="cuda"), pos // 16].long(), pos % 16)
        want, bound = ref.norm_rotate(k, None, pos, freq, False, 0)
        assert ref.close(c.k[at], want, bound, torch.bfloat16)
        assert torch.equal(c.v[at], v)


@pytest.mark.parametrize("hk,h,dim,rotary", [(8, 32, 128, 128), (4, 8, 64, 64), (1, 5, 256, 256),
                                              (8, 32, 128, 64), (3, 6, 80, 80)])
@pytest.mark.parametrize("tin,inter,norm", [("bf16", False, True), ("f32", True, True),
                                            ("bf16", True, False)])
def test_append_of_prompts(paged, hk, h, dim, rotary, tin, inter, norm):
    """Chunks of odd length, padded at their ends: a block's tokens change from padding
    to tokens, from one sequence to the next, in every place."""
    lens, chunk, q_lens = [499, 40, 700, 0, 503], 501, [499, 2, 501, 0, 3]
    c = Case(paged, 30 + dim, lens, q_lens=q_lens, kv_heads=hk, dim=dim, poison=False,
             prefix=[77], starts=[1, 4])
    rows = len(lens) * chunk
    y = randn(c.g, rows, (h + 2 * hk) * dim).to(DT[tin])
    q, k, v = (t.unflatten(1, (-1, dim)) for t in y.split([h * dim, hk * dim, hk * dim], 1))
    freq = paged.rope_frequencies(rotary, 1e4)
    w = weights(c.g, "bf16", dim) if norm else None
    k0, v0 = c.k.clone(), c.v.clone()
    out = torch.full(q.shape, math.nan, dtype=torch.bfloat16, device="cuda")
    c.kv.append(c.batch, k, v, q=q, freq=freq, q_weight=w, k_weight=w, interleaved=inter,
                q_out=out)
    i = torch.arange(chunk, device="cuda")
    real = (i < ints(q_lens)[:, None]).flatten()
    j = ((ints(lens) - ints(q_lens))[:, None] + i).flatten()
    seq = torch.arange(len(lens), device="cuda").repeat_interleave(chunk)
    pos = j + 77 * ((seq >= 1) & (seq < 4))
    want, bound = ref.norm_rotate(q, w, pos, freq, inter, 1e-6)
    assert ref.close(out[real], want[real], bound[real], torch.bfloat16) and not out[~real].any()
    at = (c.table[seq[real], j[real] // 16].long(), j[real] % 16)
    want, bound = ref.norm_rotate(k, w, pos, freq, inter, 1e-6)
    assert ref.close(c.k[at], want[real], bound[real], torch.bfloat16)
    assert torch.equal(c.v[at], v[real].bfloat16())
    c.k[at], c.v[at] = k0[at], v0[at]
    assert torch.equal(bits(c.k), bits(k0)) and torch.equal(bits(c.v), bits(v0))
    assert c.kv.device_error() == (0, 0)


def test_append_in_place(paged):
    c = Case(paged, 15, [9, 30], poison=False)
    q, k, v = (randn(c.g, 2, n, 64).bfloat16() for n in (6, 2, 2))
    freq = paged.rope_frequencies(64, 1e4)
    want, bound = ref.norm_rotate(q, None, ints([8, 29]), freq, True, 0)
    assert c.kv.append(c.batch, k, v, q=q, freq=freq, interleaved=True, q_out=q) is q
    assert ref.close(q, want, bound, torch.bfloat16)


def test_refusals_on_the_device(paged):
    """What the Python calls refuse with tensors on the device."""
    c = Case(paged, 16, [9, 30], poison=False)
    q, k, v = (randn(c.g, 2, n, 64) for n in (4, 2, 2))
    freq = paged.rope_frequencies(64, 1e4)
    append, attend = c.kv.append, c.kv.attend
    for bad in (lambda: append(c.batch, k[:1], v[:1]), lambda: append(c.batch, k, v.bfloat16()),
                lambda: append(c.batch, k, v[:, :1]), lambda: append(c.batch, k, v, q=q.half()),
                lambda: append(c.batch, k, v, q_out=q), lambda: append(c.batch, k, v, freq=freq[:30]),
                lambda: append(c.batch, k, v, q=q, q_out=q), lambda: append(c.batch, k.cpu(), v),
                lambda: append(c.batch, k, v, q_weight=torch.ones(32, device="cuda")),
                lambda: append(c.lens, k, v), lambda: attend(c.batch, q),
                lambda: attend(c.batch, q.bfloat16()[:, :3]),
                lambda: attend(c.batch, q.bfloat16()[:1]),
                lambda: attend(c.batch, torch.zeros(2 * 4 * 64 + 4, device="cuda").bfloat16()[4:]
                               .view(2, 4, 64)),
                lambda: attend(c.batch, q.bfloat16(), out=torch.empty_like(q)),
                lambda: attend(c.batch, q.bfloat16(), out=q.bfloat16()[:1].expand(2, 4, 64)),
                lambda: paged.PagedKV(c.k[:, :12], c.v[:, :12]),
                lambda: paged.PagedKV(c.k.float(), c.v.float()),
                lambda: paged.PagedKV(c.k, c.v[:1]), lambda: paged.PagedKV(c.k[..., 1:], c.v[..., 1:]),
                lambda: paged.PagedBatch(c.table, ints([1])),
                lambda: paged.PagedBatch(c.table.long(), ints([1, 2])),
                lambda: paged.PagedBatch(c.table, ints([1, 2]), prefix_table=c.table),
                lambda: paged.qk_norm_rope(q, k.bfloat16(), ints([1, 2]), freq),
                lambda: paged.qk_norm_rope(q, k, ints([1]), freq),
                lambda: paged.qk_norm_rope(q, k, ints([1, 2]), freq, out=(q, None))):
        with pytest.raises((TypeError, ValueError)):
            bad()
    leaf = q.clone().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        append(c.batch, k, v, q=leaf)
    with torch.no_grad():
        append(c.batch, k, v, q=leaf)
    assert c.kv.device_error() == (0, 0)


def test_outputs_in_other_tensors_memory_are_refused(paged):
    """Results over an input at another place, over each other or over the cache."""
    c = Case(paged, 27, [9, 30], poison=False)
    y = randn(c.g, 3, 8, 64).bfloat16()
    q, k, v = y[:2, :4], y[:2, 4:6], y[:2, 6:]
    freq, at = paged.rope_frequencies(64), ints([1, 2])
    pages = c.k.view(-1, 4, 64)[:2]
    for bad in (lambda: paged.qk_norm_rope(q, k, at, freq, out=(y[1:, :4], k)),
                lambda: paged.qk_norm_rope(k, v, at, freq, out=(v, k)),
                lambda: paged.qk_norm_rope(k, v, at, freq, out=(q[:, :2], q[:, 1:3])),
                lambda: paged.qk_norm_rope(q, k, at, freq, out=(y[:2, 2:6], y[:2, :2])),
                lambda: paged.qk_norm_rope(q.float(), None, at, freq[:4].clone(), q[0, 0],
                                           out=(q, None)),
                lambda: c.kv.append(c.batch, k, v, q=q, q_out=y[:2, 2:6]),
                lambda: c.kv.append(c.batch, k, v, q=q, q_out=pages),
                lambda: c.kv.attend(c.batch, q, out=y[1:, :4]),
                lambda: c.kv.attend(c.batch, q, out=pages)):
        with pytest.raises(ValueError, match="overlaps"):
            bad()
    k0, v0, want = c.k.clone(), v.clone(), paged.qk_norm_rope(q, k, at, freq)
    got = paged.qk_norm_rope(q, k, at, freq, out=(q, k))       # in place, beside each other
    assert got[0] is q and torch.equal(bits(q), bits(want[0]))
    assert torch.equal(bits(k), bits(want[1])) and torch.equal(bits(v), bits(v0))
    assert torch.equal(bits(c.k), bits(k0)) and c.kv.device_error() == (0, 0)


def test_append_without_q_or_rotation(paged):
    c = Case(paged, 4, [4, 9], poison=False)
    k, v = randn(c.g, 2, 2, 64), randn(c.g, 2, 2, 64)
    assert c.kv.append(c.batch, k, v) is None
    p, s = c.table[[0, 1], [0, 0]].long(), torch.tensor([3, 8], device="cuda")
    assert torch.equal(c.k[p, s], k.bfloat16()) and torch.equal(c.v[p, s], v.bfloat16())


@pytest.mark.parametrize("lens,chunk,q_lens", [
    ([0, 2, 1, 0, 5], 1, None), ([0, 2, 1, -4, 5], 3, None), ([0, 2, 1, 3, 5], 3, [0, 3, 2, 3, 1]),
    ([3] * 500, 4, None)])
def test_rows_before_a_sequences_start(paged, lens, chunk, q_lens):
    """More new tokens than a sequence has: those before its start are not appended;
    their q is that of their position, and they see the prefix, where there is one."""
    n = len(lens)
    c = Case(paged, 24, lens, q_lens=q_lens, prefix=[20, 40], starts=[0, 2, n - 1])
    q, k, v = (randn(c.g, n * chunk, h, 64) for h in (4, 2, 2))
    freq, w = paged.rope_frequencies(64, 1e4), weights(c.g, "bf16", 64)
    k0, v0 = c.k.clone(), c.v.clone()
    got = c.kv.append(c.batch, k, v, q=q, freq=freq, q_weight=w, k_weight=w)
    fresh = torch.tensor(q_lens or [chunk] * n, device="cuda")[:, None]
    i = torch.arange(chunk, device="cuda")
    j = torch.tensor(lens, device="cuda").clamp(min=0)[:, None] - fresh + i
    base = torch.tensor([20] * 2 + [40] * (n - 3) + [0], device="cuda")[:, None]
    pos, real = (base + j).flatten(), (i < fresh).flatten()
    want, bound = ref.norm_rotate(q, w, pos, freq, False, 1e-6)
    assert ref.close(got[real], want[real], bound[real], torch.bfloat16) and not got[~real].any()
    on = real & (j >= 0).flatten()
    rows, at = torch.arange(n, device="cuda").repeat_interleave(chunk)[on], j.flatten()[on]
    place = (c.table[rows, at // 16].long(), at % 16)
    want, bound = ref.norm_rotate(k, w, pos, freq, False, 1e-6)
    assert ref.close(c.k[place], want[on], bound[on], torch.bfloat16)
    assert torch.equal(c.v[place], v[on].bfloat16())
    o, lse = c.kv.attend(c.batch, got, return_lse=True)
    c.check(got, o, lse)
    c.k[place], c.v[place] = k0[place], v0[place]
    assert torch.equal(bits(c.k), bits(k0)) and torch.equal(bits(c.v), bits(v0))


def test_append_outside_the_tables(paged):
    """Pages that are not there and lengths past the table: nothing is written."""
    c = Case(paged, 5, [20, 20, 20, 20], poison=False, width=2)
    c.table[0, 1], c.table[1, 1] = -1, c.k.shape[0]
    lens = ints([20, 20, 33, 20])                      # the third's token is past its two pages
    batch = paged.PagedBatch(c.table, lens)
    k0, v0 = c.k.clone(), c.v.clone()
    q, k, v = (randn(c.g, 4, 2, 64) for _ in range(3))
    got = c.kv.append(batch, k, v, q=q)
    assert torch.equal(got, q.bfloat16())
    assert torch.equal(c.k[c.table[3, 1], 3], k[3].bfloat16())
    c.k[c.table[3, 1], 3], c.v[c.table[3, 1], 3] = k0[c.table[3, 1], 3], v0[c.table[3, 1], 3]
    assert torch.equal(bits(c.k), bits(k0)) and torch.equal(bits(c.v), bits(v0))
    assert c.kv.device_error() == (1, 4) and c.kv.device_error() == (0, 0)
    # A length of fewer than the new tokens leaves those before the start out.
    c.kv.append(paged.PagedBatch(c.table, ints([0, -3, 0, 0])), k, v)
    assert torch.equal(bits(c.k), bits(k0)) and c.kv.device_error() == (0, 0)


# ---- attention --------------------------------------------------------------

ATTEND = [  # lens, chunk, q_lens, heads, kw
    ([1], 1, None, 2, {}),
    ([127], 1, None, 8, dict(dim=128)),
    ([128, 129, 255, 256, 257], 1, None, 4, {}),
    ([1003], 1, None, 32, dict(kv_heads=8, dim=128)),
    ([5000], 1, None, 8, dict(kv_heads=1, dim=128, page=8)),
    ([0, 3, 0, 70], 1, None, 2, dict(page=8)),
    ([0, 0], 1, None, 2, {}),
    ([3, 300, 12, 9, 1], 1, None, 6, dict(prefix=[100, 700], starts=[1, 3, 4])),
    ([1] * 8, 1, None, 32, dict(kv_heads=8, dim=128, prefix=[777], starts=[0, 8])),
    ([7, 0, 20, 1], 1, None, 4, dict(prefix=[0, 31, 50], starts=[0, 1, 1, 4])),
    ([9, 33, 2], 2, None, 4, dict(page=64)),
    ([40, 23, 64], 20, [20, 3, 0], 2, dict(page=32, dim=128)),
    ([66, 70], 66, [2, 66], 14, dict(prefix=[1000], starts=[0, 2], heads_first=True, dim=128)),
    ([200], 200, None, 2, dict(page=16)),
    ([700, 333], 150, [150, 77], 8, dict(page=256, prefix=[129, 5], starts=[0, 1, 2])),
    ([17] * 64, 1, None, 8, dict(prefix=[2500], starts=[0, 64])),
    ([17] * 64, 1, None, 32, dict(kv_heads=8, dim=128, prefix=[600], starts=[0, 64])),
    ([4] * 70, 1, None, 16, dict(kv_heads=1, prefix=[300, 40], starts=[0, 68, 70])),
    ([31] * 130, 1, None, 2, dict(prefix=[64] * 65, starts=list(range(0, 131, 2)))),
    ([9] * 500, 1, None, 1, dict(kv_heads=1, prefix=[20, 20], starts=[0, 100, 400], page=8)),
    ([2, 1, 3], 3, [2, 1, 3], 10, dict(prefix=[128], starts=[0, 3], dim=128)),
    ([100, 20], 1, None, 128, dict(kv_heads=1, dim=128)),
    ([300], 3, None, 256, dict(kv_heads=2, dim=64)),
    ([20000], 64, None, 8, dict(kv_heads=2, dim=128, page=64)),
    # Heads that come by eight, four, two and one to a tile, rows up to and over 16.
    ([130, 1, 17, 300], 1, None, 48, dict(kv_heads=16, page=8)),
    ([130, 0, 17, 300], 3, [3, 1, 2, 3], 24, dict(kv_heads=12, dim=128, page=128)),
    ([900, 64, 33], 1, None, 72, dict(kv_heads=6, page=16, prefix=[65], starts=[1, 3])),
    ([900, 64, 33], 4, None, 12, dict(kv_heads=3, dim=128, page=8, prefix=[131], starts=[0, 2])),
    ([500, 77], 1, None, 12, dict(kv_heads=1, dim=128, page=64)),
    ([500, 77], 17, [17, 5], 3, dict(kv_heads=3, page=32)),
    ([1300], 5, None, 13, dict(kv_heads=1, page=16, prefix=[3], starts=[0, 1])),
    ([33, 65, 129] * 3, 1, None, 8, dict(kv_heads=8, dim=128, page=256)),
    # Long and short shares of every kind of rows in turn, many parts an SM.
    ([7 * i % 500 + 1 for i in range(64)], 1, None, 32,
     dict(kv_heads=8, dim=128, prefix=[8200], starts=[0, 64])),
    ([11 * i % 900 for i in range(90)], 1, None, 16,
     dict(kv_heads=4, prefix=[3000, 5000, 700, 2600, 4000, 900], starts=[0, 2, 70, 74, 85, 86, 90])),
    ([11 * i % 900 for i in range(90)], 1, None, 16,
     dict(kv_heads=4, dim=128, prefix=[3000, 5000, 700, 2600, 4000, 900],
          starts=[0, 2, 70, 74, 85, 86, 90])),
    ([257] * 140, 3, None, 16, dict(kv_heads=4, dim=128, prefix=[1500] * 4,
                                    starts=[0, 30, 35, 36, 140])),
]


@pytest.mark.parametrize("lens,chunk,q_lens,heads,kw", ATTEND)
def test_attend(paged, lens, chunk, q_lens, heads, kw):
    c = Case(paged, len(lens) + heads, lens, q_lens=q_lens, **kw)
    q = (2 * randn(c.g, len(lens) * chunk, heads, c.kv.dim)).bfloat16()
    got, lse = c.kv.attend(c.batch, q, return_lse=True)
    c.check(q, got, lse)
    again = c.kv.attend(c.batch, q)
    assert torch.equal(bits(got), bits(again))          # the same bits on every run


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_attend_scales(paged, scale):
    """Uniform weights, turned signs, and scores of hundreds (one token takes all)."""
    c = Case(paged, 6, [500, 40], dim=128, prefix=[900], starts=[0, 2])
    q = (3 * randn(c.g, 2, 4, 128)).bfloat16()
    got, lse = c.kv.attend(c.batch, q, scale=scale, return_lse=True)
    c.check(q, got, lse, scale)


@pytest.mark.parametrize("chunk,heads", [(1, 1), (3, 8), (40, 4)])
@pytest.mark.parametrize("scale", [0.0, 1e-45, -1e-40, 2.0 ** -120])
def test_attend_tiny_scales(paged, chunk, heads, scale):
    """Scales near and at zero with products near FP32's largest: a scale of zero weighs
    every token alike, whatever its product."""
    c = Case(paged, 26, [60, 300], kv_heads=1, dim=64, prefix=[200], starts=[0, 1])
    q = torch.zeros((2 * chunk, heads, 64), device="cuda").bfloat16()
    c.k[torch.isfinite(c.k)] *= 2.0 ** -20
    q[..., 0] = 2.0 ** 62
    for row, n in ((c.table[0], 60), (c.table[1], 300), (c.far[0], 200)):
        at = torch.arange(0, n, 3, device="cuda")
        c.k[row[at // 16].long(), at % 16, :, 0] = 2.0 ** 64      # products of 2^126
    got, lse = c.kv.attend(c.batch, q, scale=scale, return_lse=True)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    want, bound, want_lse, lse_bound = c.want(q, scale)
    # The least FP32 number as scale moves a weight by less than 2^-20 of itself.
    size = torch.nan_to_num(c.v.float(), 0, 0, 0).abs().max()
    assert ref.close(got, want, bound + 2.0 ** -19 * size, torch.bfloat16)
    assert bool(((lse.double() - want_lse).abs() <= lse_bound + 2.0 ** -19).all())
    assert c.kv.device_error() == (0, 0)


def test_attend_rising_scores(paged):
    """A running maximum that grows by more than any fixed step tile after tile."""
    c = Case(paged, 7, [1500], kv_heads=1, dim=64, prefix=[1024], starts=[0, 1])
    step = torch.linspace(0, 40, 1024, device="cuda").bfloat16()
    flat = c.far[0, :64].long()
    c.k[flat] = step.view(64, 16, 1, 1).expand(64, 16, 1, 64)
    q = torch.full((1, 2, 64), 1.0, device="cuda").bfloat16()
    q[0, 1] = -1
    got, lse = c.kv.attend(c.batch, q, return_lse=True)
    c.check(q, got, lse)


def test_attend_infinite_keys(paged):
    """Keys that make scores of -inf for some rows: such tokens weigh nothing; a
    row with no other token is zero with an lse of -inf."""
    c = Case(paged, 8, [300, 16], kv_heads=1, dim=64, poison=False)
    q = torch.zeros((2, 1, 64), device="cuda").bfloat16()
    q[..., 0] = 1
    for b, n in ((0, 300), (1, 16)):
        pages = c.table[b, :-(-n // 16)].long()
        c.k[pages, :, :, 0] = 1.0
    c.k[c.table[0, :10].long(), :, :, 0] = -math.inf
    c.k[c.table[1, 0].long(), :, :, 0] = -math.inf
    got, lse = c.kv.attend(c.batch, q, return_lse=True)
    live = c.v[c.table[0, 10:19].long()].flatten(0, 1)[:140].double()
    assert (got[0].double() - live.mean(0)).abs().max() <= 2.0 ** -7 * live.abs().max()
    assert abs(float(lse[0, 0]) - (math.log(140) + 0.125)) < 1e-4
    assert not got[1].any() and lse[1, 0] == -math.inf


@pytest.mark.parametrize("lens,chunk,q_lens,heads,kw", [
    ([40, 9, 7], 3, [3, 2, 3], 4, {}),
    ([150, 33], 8, None, 8, dict(kv_heads=8, dim=128, prefix=[70], starts=[0, 1])),
    ([300, 20], 20, [20, 12], 8, dict(prefix=[129], starts=[0, 2], page=32, dim=128)),
    ([400], 200, None, 2, dict(kv_heads=1, page=8))])
@pytest.mark.parametrize("scale", [0.125, -0.2])
def test_attend_values_that_are_not_finite(paged, lens, chunk, q_lens, heads, kw, scale):
    """An infinite or NaN V reaches the rows that see its token, and no other."""
    c = Case(paged, 21, lens, q_lens=q_lens, **kw)
    dim = c.k.shape[3]
    for b, n in enumerate(lens):
        fresh = chunk if q_lens is None else q_lens[b]
        for back, d, x in ((1, 0, math.inf), (2, 5, math.nan), (fresh // 2 + 1, 9, -math.inf),
                           (fresh // 2 + 1, dim - 1, math.inf)):
            if back <= fresh:
                page = c.k.shape[1]
                c.v[c.table[b, (n - back) // page].long(), (n - back) % page, b % c.k.shape[2], d] = x
    q = randn(c.g, len(lens) * chunk, heads, dim).bfloat16()
    got, lse = c.kv.attend(c.batch, q, scale=scale, return_lse=True)
    want, bound, want_lse, lse_bound = c.want(q, scale)
    fine = torch.isfinite(want)
    assert not fine.all()
    assert ref.close(got[fine], want[fine], bound[fine], torch.bfloat16)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)].double(), want[torch.isinf(want)])
    seen = torch.isfinite(want_lse)
    assert bool(((lse.double() - want_lse).abs()[seen] <= lse_bound[seen]).all())
    assert c.kv.attend(c.batch, q, out=q, scale=scale) is q     # in place, to the bit
    assert torch.equal(bits(q), bits(got)) and c.kv.device_error() == (0, 0)


def test_attend_values_that_are_not_finite_cost_nothing(paged):
    """Not finite in tokens that every row sees: the same answer in the same time, to a
    factor that tells it from a second pass over the context."""
    c = Case(paged, 25, [40] * 4, prefix=[30000], starts=[0, 4], dim=128)
    q = randn(c.g, 4 * 8, 8, 128).bfloat16()

    def least():
        took = []
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            c.kv.attend(c.batch, q)
            b.record()
            b.synchronize()
            took.append(a.elapsed_time(b))
        return min(took)

    clean = least()
    c.v[c.far[0, 3].long(), 5, :, 7] = math.nan
    c.v[c.table[1, 0].long(), 2, 0] = math.inf
    got = c.kv.attend(c.batch, q)
    want, bound, _, _ = c.want(q, 128 ** -0.5)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and not fine.all()
    assert ref.close(got[fine], want[fine], bound[fine], torch.bfloat16)
    assert least() < 4 * clean and c.kv.device_error() == (0, 0)


@pytest.mark.parametrize("lens,chunk,heads,kw", [
    ([40, 9], 3, 4, {}), ([300, 20], 20, 8, dict(prefix=[129], starts=[0, 2], dim=128)),
    ([400], 200, 2, dict(kv_heads=1, page=8))])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attend_keys_that_are_not_finite(paged, lens, chunk, heads, kw, bad):
    """So does such a K: the rows before its token are right."""
    c = Case(paged, 22, lens, **kw)
    page, back = c.k.shape[1], chunk // 2
    for b, n in enumerate(lens):
        c.k[c.table[b, (n - back) // page].long(), (n - back) % page, :, 3] = bad
    q = randn(c.g, len(lens) * chunk, heads, c.k.shape[3]).bfloat16()
    got, lse = c.kv.attend(c.batch, q, return_lse=True)
    want, bound, want_lse, lse_bound = c.want(q, c.k.shape[3] ** -0.5)
    before = (torch.arange(chunk, device="cuda") < chunk - back).repeat(len(lens))
    assert torch.isfinite(want[before]).all()
    assert ref.close(got[before], want[before], bound[before], torch.bfloat16)
    assert bool(((lse.double() - want_lse).abs()[before] <= lse_bound[before]).all())
    if math.isnan(bad):
        assert torch.isnan(got[~before]).all()
    assert c.kv.device_error() == (0, 0)


def test_attend_missing_pages(paged):
    """A page outside the pool counts as zeros and is reported, tokens past the
    table are not seen."""
    c = Case(paged, 9, [64, 64], poison=False, width=4)
    c.table[0, 2] = c.k.shape[0] + 5
    q = randn(c.g, 2, 2, 64).bfloat16()
    got = c.kv.attend(c.batch, q)
    assert c.kv.device_error() == (1, 4)
    k = torch.cat((c.k, torch.zeros_like(c.k[:1])))
    v = torch.cat((c.v, torch.zeros_like(c.v[:1])))
    table = c.table.clone()
    table[0, 2] = c.k.shape[0]
    want, bound, _, _ = ref.attention(q, k, v, table, [64, 64], None, None, None, None, 1 / 8)
    assert ref.close(got, want, bound, torch.bfloat16)
    over = paged.PagedBatch(c.table[1:], ints([90]))
    got = c.kv.attend(over, q[1:])
    assert c.kv.device_error() == (1, 4)
    assert ref.close(got, want[1:], bound[1:], torch.bfloat16)


def test_attend_bounded_waits(paged):
    """With a limit of one poll the kernel's waits give up: it returns, says so, and
    the next call is right."""
    from lossless_bf16_weight_nwc_b200 import _lib
    c = Case(paged, 12, [300] * 6, dim=128, kv_heads=4, prefix=[900], starts=[0, 6])
    q = randn(c.g, 6, 32, 128).bfloat16()
    _lib.nwc_test_set_wait_limit(1)
    try:
        c.kv.attend(c.batch, q)
        status, word = c.kv.device_error()
    finally:
        _lib.nwc_test_set_wait_limit(0)
    assert (status, word & 1) == (6, 1)                  # NWC_ERR_DEVICE_TIMEOUT
    got, lse = c.kv.attend(c.batch, q, return_lse=True)
    c.check(q, got, lse)


@pytest.mark.parametrize("limit", [1, 30, 300])
@pytest.mark.parametrize("lens,chunk,heads,kw", [
    ([400] * 3, 150, 8, dict(kv_heads=4, dim=128, prefix=[900], starts=[0, 3])),   # both teams
    ([700] * 12, 1, 32, dict(kv_heads=2, prefix=[1500, 300], starts=[0, 9, 11])),  # every kind
    ([2000], 64, 8, dict(kv_heads=4, page=64))])                                   # one team
def test_attend_bounded_waits_of_every_kind(paged, limit, lens, chunk, heads, kw):
    """Waits that give up at the first poll or further on, in parts of every kind of
    rows: the kernel returns, and the next call is right."""
    from lossless_bf16_weight_nwc_b200 import _lib
    c = Case(paged, 23, lens, **kw)
    q = randn(c.g, len(lens) * chunk, heads, c.kv.dim).bfloat16()
    _lib.nwc_test_set_wait_limit(limit)
    try:
        for _ in range(3):
            c.kv.attend(c.batch, q)
        status, word = c.kv.device_error()
    finally:
        _lib.nwc_test_set_wait_limit(0)
    assert (status, word) in ((6, 1), (0, 0)) and (word or limit > 1)
    got, lse = c.kv.attend(c.batch, q, return_lse=True)
    c.check(q, got, lse)


def test_attend_tables_without_columns_after_others(paged):
    """Lengths that no table holds leave nothing to see, whatever an earlier call of
    the same shape left in the workspace."""
    from lossless_bf16_weight_nwc_b200 import _lib
    c = Case(paged, 19, [40, 30], prefix=[50], starts=[0, 2], poison=False)
    q = randn(c.g, 2, 4, 64).bfloat16()
    none = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    shared = (ints(c.prefix), ints(c.starts))
    empty = paged.PagedBatch(none, ints(c.lens), None, none[:1], *shared)
    own = paged.PagedBatch(c.table, ints(c.lens), None, none[:1], *shared)
    need = [_lib.nwc_kv_attention_workspace(c.kv._view, _lib.nwc_kv_batch.from_address(b._view(2)), 4)
            for b in (c.batch, empty)]
    assert need[0] == need[1]
    ws = torch.zeros(need[0], dtype=torch.uint8, device="cuda")

    def attend(batch):
        out, lse = torch.full_like(q, 7.0), torch.full((2, 4), 7.0, device="cuda")
        view = [_lib.nwc_heads.from_buffer_copy(paged._heads(t, "t", t.shape, t.device))
                for t in (q, out)]
        _lib.nwc_kv_attention(c.kv._view, _lib.nwc_kv_batch.from_address(batch._view(2)), view[0],
                              4, 1 / 8, view[1], lse, ws, need[0])
        return out, lse

    c.check(q, *attend(c.batch))
    out, lse = attend(empty)
    assert not out.any() and bool((lse == -math.inf).all())
    assert c.kv.device_error() == (1, 4)
    attend(c.batch)
    want, bound, _, _ = ref.attention(q, c.k, c.v, c.table, c.lens, None, None, None, None, 1 / 8)
    assert ref.close(attend(own)[0], want, bound, torch.bfloat16)
    assert c.kv.device_error() == (1, 4)


def test_gradients_are_refused_everywhere(paged):
    """Every tensor of a call that requires a gradient, results' own included."""
    from lossless_bf16_weight_nwc_b200 import _lib, synth
    c = Case(paged, 20, [9, 30], poison=False)
    q, k, v = (randn(c.g, 2, n, 64).bfloat16() for n in (4, 2, 2))
    freq, at, w = paged.rope_frequencies(64), ints([1, 2]), torch.ones(64, device="cuda")
    eye = [synth.matrix(synth.MatrixSpec("w", r, 256, "normal", 0.06, 0), 1)
           for r in (256, 128, 128, 256)]
    block = paged.AttentionBlock(_lib.CompressedMatrix.compress_fused(eye[:3]),
                                 _lib.CompressedMatrix.compress(eye[3]), c.kv, freq)
    x = randn(c.g, 2, 256).bfloat16()
    calls = [(lambda t: paged.qk_norm_rope(t, k, at, freq), q),
             (lambda t: paged.qk_norm_rope(q, k, at, t), freq),
             (lambda t: paged.qk_norm_rope(q, k, at, freq, t), w),
             (lambda t: paged.qk_norm_rope(q, None, at, freq, out=(t, None)), q),
             (lambda t: c.kv.append(c.batch, t, v), k), (lambda t: c.kv.append(c.batch, k, t), v),
             (lambda t: c.kv.append(c.batch, k, v, freq=t), freq),
             (lambda t: c.kv.append(c.batch, k, v, q=q, q_out=t), q),
             (lambda t: c.kv.attend(c.batch, t), q),
             (lambda t: c.kv.attend(c.batch, q, out=t), q),
             (lambda t: block.step(t, c.batch), x)]
    k0, v0 = bits(c.k), bits(c.v)
    for call, t in calls:
        with pytest.raises(ValueError, match="gradient"):
            call(t.clone().requires_grad_())
    assert torch.equal(bits(c.k), k0) and torch.equal(bits(c.v), v0)
    with torch.no_grad():
        for call, t in calls:
            call(t.clone().requires_grad_())
    assert c.kv.device_error() == (0, 0)


def test_pages_that_come_to_require_a_gradient(paged):
    c = Case(paged, 28, [9, 30], poison=False)
    q, k, v = (randn(c.g, 2, n, 64).bfloat16() for n in (4, 2, 2))
    k0 = bits(c.k)
    for pages in (c.k, c.v):
        pages.requires_grad_()
        for call in (lambda: c.kv.append(c.batch, k, v), lambda: c.kv.attend(c.batch, q)):
            with pytest.raises(ValueError, match="gradient"):
                call()
        pages.requires_grad_(False)
    assert torch.equal(bits(c.k), k0)
    c.k.requires_grad_()
    with torch.no_grad():
        c.kv.append(c.batch, k, v)
        got = c.kv.attend(c.batch, q)
    c.k.requires_grad_(False)
    c.check(q, got)


def test_attend_unordered_groups(paged):
    """Group starts that are not ascending or point outside: some answer, nothing
    written out of bounds, and the rows outside such groups are right."""
    c = Case(paged, 13, [40] * 8, prefix=[500, 300, 100], starts=[0, 2, 4, 8])
    q = randn(c.g, 8, 4, 64).bfloat16()
    for starts in ([4, 2, 9, 1], [-3, 0, 100, 100], [8, 8, 8, 8], [0, 8, 0, 8]):
        batch = paged.PagedBatch(c.table, ints(c.lens), None, c.far, ints(c.prefix), ints(starts))
        out = torch.full((10, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        c.kv.attend(batch, q, out=out[1:9])
        assert bool((out[[0, 9]] == 7).all())
        c.kv.device_error()
    got, lse = c.kv.attend(c.batch, q, return_lse=True)
    c.check(q, got, lse)


def attend_c(paged, c, batch, q, chunk=1):
    """(out, lse) through the C call's own structures, with a workspace of the stated size
    between bytes that have to stay."""
    from lossless_bf16_weight_nwc_b200 import _lib
    rows, heads, dim = q.shape
    view = _lib.nwc_kv_batch.from_address(batch._view(rows))
    need = _lib.nwc_kv_attention_workspace(c.kv._view, view, heads)
    ws = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((rows, heads), 7.0, device="cuda")
    qv, ov = (_lib.nwc_heads.from_buffer_copy(paged._heads(t, "t", t.shape, t.device))
              for t in (q, out))
    _lib.nwc_kv_attention(c.kv._view, view, qv, heads, dim ** -0.5, ov, lse, ws[4096:], need)
    assert bool((ws[:4096] == 0xA5).all()) and bool((ws[4096 + need:] == 0xA5).all())
    return out, lse


@pytest.mark.parametrize("starts", [[4, 2, 9, 1], [-3, 0, 100, 100], [8, 8, 8, 8], [0, 8, 0, 8],
                                    [2, 5, 5, 5], [0, 0, 0, 8], [9, -1, 3, 2]])
@pytest.mark.parametrize("chunk,heads", [(1, 4), (5, 8), (40, 8)])
def test_attend_unordered_groups_values(paged, starts, chunk, heads):
    """Group starts out of order or outside: sequences that no group holds have no
    prefix, those that one group holds have its, and nothing is written elsewhere."""
    c = Case(paged, 32, [40] * 8, prefix=[500, 300, 100], starts=[0, 2, 4, 8])
    q = randn(c.g, 8 * chunk, heads, 64).bfloat16()
    batch = paged.PagedBatch(c.table, ints(c.lens), None, c.far, ints(c.prefix), ints(starts))
    out, lse = attend_c(paged, c, batch, q)
    held = [[g for g in range(3) if starts[g] <= b < starts[g + 1]] for b in range(8)]
    for b, groups in enumerate(held):
        rows = slice(b * chunk, (b + 1) * chunk)
        if len(groups) < 2:
            far = (c.far[groups], [c.prefix[groups[0]]], [0, 1]) if groups else (None, None, None)
            want, bound, want_lse, lse_bound = ref.attention(
                q[rows], c.k, c.v, c.table[b:b + 1], [40], None, *far, 1 / 8)
            assert ref.close(out[rows], want, bound, torch.bfloat16)
            assert bool(((lse[rows].double() - want_lse).abs() <= lse_bound).all())
    # Two groups over 1280 rows of a key head are 5 blocks x 2 heads each: 20 items, where
    # the workspace of 1280 rows and 3 groups has (5 + 3) x 2.
    overlap = any(len(groups) > 1 for groups in held)
    assert c.kv.device_error() == ((1, 4) if overlap and chunk == 40 else (0, 0))


def test_attend_groups_that_overlap(paged):
    """More rows in groups than there are rows: reported, nothing written elsewhere,
    and the next call is right."""
    n = 128
    c = Case(paged, 33, [9] * n, prefix=[200] * 8, starts=[16 * i for i in range(9)])
    q = randn(c.g, n, 16, 64).bfloat16()
    batch = paged.PagedBatch(c.table, ints(c.lens), None, c.far, ints(c.prefix),
                             ints([0, n] * 4 + [0]))
    attend_c(paged, c, batch, q)
    assert c.kv.device_error() == (1, 4)
    c.check(q, *attend_c(paged, c, c.batch, q))


def test_typed_calls(paged):
    """The C calls with _lib's structures give what the Python calls do."""
    from lossless_bf16_weight_nwc_b200 import _lib
    c = Case(paged, 34, [9, 30], poison=False)
    q, k, v = (randn(c.g, 2, n, 64) for n in (4, 2, 2))
    freq, at, w = paged.rope_frequencies(64), ints([8, 29]), weights(c.g, "f32", 64)

    def view(t):
        return _lib.nwc_heads.from_buffer_copy(paged._heads(t, "t", t.shape, t.device))

    rope = _lib.nwc_rope.from_buffer_copy(paged._rope(64, q.device, freq, w, w, 1e-6, True))
    batch = _lib.nwc_kv_batch.from_address(c.batch._view(2))
    want = paged.qk_norm_rope(q, k, at, freq, w, w, interleaved=True)
    got = [torch.empty_like(t) for t in want]
    _lib.nwc_qk_norm_rope(view(q), view(k), view(got[0]), view(got[1]), 2, 4, 2, 64, at, False,
                          rope)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    rotated = torch.empty_like(got[0])
    _lib.nwc_kv_append(c.kv._view, batch, view(q), view(rotated), 4, view(k), view(v), rope)
    assert torch.equal(rotated, got[0])
    place = c.table[[0, 1], [0, 1]].long(), torch.tensor([8, 13], device="cuda")
    assert torch.equal(c.k[place], got[1]) and torch.equal(c.v[place], v.bfloat16())
    out, lse = attend_c(paged, c, c.batch, rotated)
    assert torch.equal(out, c.kv.attend(c.batch, rotated))
    c.check(rotated, out, lse)
    assert _lib.nwc_kv_get_error(c.kv._view) == (0, 0)


def test_attend_shared_pages_and_repeats(paged):
    """Sequences that point at the same pages, and a prefix whose pages repeat."""
    c = Case(paged, 14, [64, 64, 64], prefix=[64], starts=[0, 3], poison=False)
    c.table[1] = c.table[0]
    c.table[2, :4] = c.table[0, 0]
    c.far[0, :4] = c.far[0, 1]
    q = randn(c.g, 3, 8, 64).bfloat16()
    got, lse = c.kv.attend(c.batch, q, return_lse=True)
    c.check(q, got, lse)


def test_attend_strides(paged):
    c = Case(paged, 10, [50, 7, 80], kv_heads=2, dim=64, heads_first=True)
    q = randn(c.g, 4, 3, 128).bfloat16()[..., 64:].transpose(0, 1)     # heads outside tokens
    store = torch.zeros((3, 5, 72), dtype=torch.bfloat16, device="cuda")
    out = store[:, 1:, 8:]
    assert c.kv.attend(c.batch, q, out=out) is out
    c.check(q, out)
    assert not store[:, 0].any() and not store[..., :8].any()


@pytest.mark.parametrize("layout", ["K beside V", "gaps", "heads outside", "V is K", "large pages"])
def test_page_layouts(paged, layout):
    """Pages that are views: of one tensor for K and V, with gaps between heads and
    tokens, with heads outside pages, the same tensor twice, pages longer than a tile."""
    g, page, hk, dim = gen(50), 16, 3, 64
    if layout == "K beside V":
        k, v = randn(g, 30, 2, page, hk, dim).bfloat16().unbind(1)
    elif layout == "gaps":
        k, v = (randn(g, 30, page + 1, hk + 2, dim + 8).bfloat16()[:, :page, 1:hk + 1, 8:]
                for _ in range(2))
    elif layout == "heads outside":
        k, v = (randn(g, hk, 30, page, dim).bfloat16().permute(1, 2, 0, 3) for _ in range(2))
    elif layout == "V is K":
        k = v = randn(g, 30, page, hk, dim).bfloat16()
    else:
        page = 4096
        k, v = (randn(g, 4, page, hk, dim).bfloat16() for _ in range(2))
    pool = paged.PagedKV(k, v)
    own = (torch.randperm(k.shape[0], generator=g, device="cuda").int()
           if page > 16 else torch.randperm(30, generator=g, device="cuda").int()[:28])
    table, far = (own[:2].view(2, 1), own[2:].view(1, 2)) if page > 16 else (
        own[:20].view(2, 10), own[20:].view(1, 8))
    lens, prefix = ([3000, 129], [4099]) if page > 16 else ([155, 17], [120])
    batch = paged.PagedBatch(table, ints(lens), None, far, ints(prefix), ints([0, 2]))
    new = [randn(g, 4, hk, dim) for _ in range(2)]
    k0, v0 = k.clone(), v.clone()
    if layout != "V is K":
        pool.append(batch, *new)
        for b, n in enumerate(lens):
            for i in range(2):
                at = int(table[b, (n - 2 + i) // page]), (n - 2 + i) % page
                k0[at], v0[at] = new[0][2 * b + i].bfloat16(), new[1][2 * b + i].bfloat16()
        assert torch.equal(k, k0) and torch.equal(v, v0)
    for heads, chunk in ((3, 1), (12, 2), (24, 40 if page > 16 else 17)):
        q = randn(g, 2 * chunk, heads, dim).bfloat16()
        got, lse = pool.attend(batch, q, return_lse=True)
        want, bound, want_lse, lse_bound = ref.attention(q, k, v, table, lens, None, far, prefix,
                                                         [0, 2], 1 / 8)
        assert ref.close(got, want, bound, torch.bfloat16)
        assert bool(((lse.double() - want_lse).abs() <= lse_bound).all())
    assert pool.device_error() == (0, 0)


@pytest.mark.parametrize("heads,kw", [(1, dict(kv_heads=1)), (8, dict(kv_heads=2, dim=128))])
def test_attend_many_sequences_and_groups(paged, heads, kw):
    """More segments than a CTA's first look at them holds, empty groups among them."""
    n, groups = 2600, 900
    starts = [0] + sorted((i * 7919) % n for i in range(groups - 1)) + [n]
    c = Case(paged, 51, [(i * 37) % 50 for i in range(n)], page=8,
             prefix=[(i * 53) % 70 for i in range(groups)], starts=starts, **kw)
    q = randn(c.g, n, heads, c.kv.dim).bfloat16()
    got, lse = c.kv.attend(c.batch, q, return_lse=True)
    c.check(q, got, lse)


@pytest.mark.parametrize("own,far,chunk", [(2 ** 20 + 3, 0, 1), (5, 2 ** 20 + 77, 1),
                                           (2 ** 19 + 1, 2 ** 19, 33)])
def test_attend_long(paged, own, far, chunk):
    """A million tokens: sums of 2^20 terms over all CTAs."""
    kw = dict(prefix=[far], starts=[0, 1]) if far else {}
    c = Case(paged, 52, [own], kv_heads=1, page=64, **kw)
    q = (2 * randn(c.g, chunk, 2, 64)).bfloat16()
    got, lse = c.kv.attend(c.batch, q, return_lse=True)
    want, bound, want_lse, lse_bound = c.want(q, 1 / 8)
    assert ref.close(got, want, bound, torch.bfloat16)
    # 64 sums in a tile, 56 tiles a CTA, up to 300 parts: 420 roundings of 2^-24.
    assert bool(((lse.double() - want_lse).abs() <= lse_bound + 2.0 ** -15).all())
    assert c.kv.device_error() == (0, 0)


def test_attend_far_offsets(paged):
    """Pages whose offsets pass 2^32 elements."""
    pages, page, hk, dim = 70000, 128, 8, 64
    k = torch.empty((pages, page, hk, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 32
    g = gen(11)
    ids = [pages - 1, 3, pages - 77, 65540]
    for i in ids:
        k[i], v[i] = randn(g, page, hk, dim).bfloat16(), randn(g, page, hk, dim).bfloat16()
    kv = paged.PagedKV(k, v)
    table = ints([ids])
    batch = paged.PagedBatch(table, ints([400]))
    new = [randn(g, 1, hk, dim) for _ in range(2)]
    kv.append(batch, *new)
    assert torch.equal(k[65540, 15], new[0][0].bfloat16())
    assert torch.equal(v[65540, 15], new[1][0].bfloat16())
    q = randn(g, 1, 16, dim).bfloat16()
    got = kv.attend(batch, q)
    want, bound, _, _ = ref.attention(q, k, v, table, [400], None, None, None, None, 1 / 8)
    assert ref.close(got, want, bound, torch.bfloat16) and kv.device_error() == (0, 0)


# ---- streams, graphs, the run of all three ------------------------------------

def test_other_streams_at_once(paged):
    """Two batches at once, on streams that are not the current one."""
    cases = [Case(paged, 20 + i, [300 + i] * 12, dim=128, prefix=[3000], starts=[0, 12])
             for i in range(2)]
    qs = [randn(c.g, 12, 8, 128).bfloat16() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, c in enumerate(cases):
            got[i].append(c.kv.attend(c.batch, qs[i], stream=streams[i]))
    one = cases[0].kv.attend(cases[0].batch, qs[0], stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(bits(one), bits(got[0][0]))
    for i, c in enumerate(cases):
        for o in got[i]:
            assert torch.equal(bits(o), bits(got[i][0]))
        c.check(qs[i], got[i][0])


def test_calls_from_several_threads(paged):
    """The first calls of a process included: each thread on a stream of its own, over
    one cache and one batch."""
    import threading
    c = Case(paged, 29, [200, 31, 7], dim=128, kv_heads=4, prefix=[500], starts=[0, 2])
    one = {n: randn(c.g, 3 * n, 8, 128).bfloat16() for n in (1, 2, 5)}
    c.batch = paged.PagedBatch(*c.batch._keep)
    torch.cuda.synchronize()
    got, failed = {}, []

    def work(i):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                for n in (1, 2, 5, 1):
                    o = c.kv.attend(c.batch, one[n])
                    r, _ = paged.qk_norm_rope(one[n], None, at[:3 * n], freq)
                    torch.cuda.current_stream().synchronize()
                    got[i, n] = (o, r)
        except Exception as e:      # noqa: BLE001 (a thread's error, shown below)
            failed.append(e)

    freq, at = paged.rope_frequencies(128), torch.arange(15, device="cuda")
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for n in one:
        want = c.kv.attend(c.batch, one[n]), paged.qk_norm_rope(one[n], None, at[:3 * n], freq)[0]
        for i in range(6):
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got[i, n], want))
        c.check(one[n], want[0])


def test_other_streams_for_every_call(paged):
    """The stream given and a current stream that is not the default: results are
    allocated there, an eager run beside a captured and replayed one."""
    g = gen(31)
    pool = paged.PagedKV(*(randn(g, 9, 16, 2, 64).bfloat16() for _ in range(2)))
    batch = paged.PagedBatch(torch.arange(8, device="cuda").int().view(2, 4), ints([5, 40]))
    q, k, v = (randn(g, 2, n, 64) for n in (4, 2, 2))
    freq, at = paged.rope_frequencies(64), ints([4, 39])

    def run(stream=None):
        a, b = paged.qk_norm_rope(q, k, at, freq, stream=stream)
        c = pool.append(batch, k, v, q=q, freq=freq, stream=stream)
        return a, b, c, *pool.attend(batch, c, return_lse=True, stream=stream)

    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [run(side), run(side.cuda_stream)]
    with torch.cuda.stream(side):
        got.append(run())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(run())
    with torch.cuda.stream(side):
        got.append(run())
    graph.replay()
    torch.cuda.synchronize()
    for other in got:
        assert all(torch.equal(x, y) for x, y in zip(other, want))
    assert pool.device_error(side) == (0, 0)


def test_graph_replays_follow_lengths(paged):
    """A captured append + attend replayed as the sequences grow; two graphs of
    one cache keep their own workspace."""
    g = gen(30)
    pool = paged.PagedKV(randn(g, 40, 16, 2, 64).bfloat16(), randn(g, 40, 16, 2, 64).bfloat16())
    table = torch.randperm(40, generator=g, device="cuda").int()[:37].contiguous()
    own, far = table[:24].view(3, 8), table[24:].view(1, 13)
    lens = ints([1, 20, 47])
    batch = paged.PagedBatch(own, lens, prefix_table=far, prefix_lens=ints([200]),
                             group_start=ints([0, 2]))
    freq = paged.rope_frequencies(64, 1e4)
    q, k, v = (randn(g, 3, n, 64) for n in (4, 2, 2))

    def step():
        qr = pool.append(batch, k, v, q=q, freq=freq)
        return qr, pool.attend(batch, qr)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        graphs.append((graph, outs))
    now = [1, 20, 47]
    for turn in range(30):
        q.copy_(randn(g, 3, 4, 64)), k.copy_(randn(g, 3, 2, 64)), v.copy_(randn(g, 3, 2, 64))
        graph, (qr, o) = graphs[turn % 2]
        graph.replay()
        want, bound, _, _ = ref.attention(qr, pool.k_pages, pool.v_pages, own, now, None, far,
                                          [200], [0, 2], 1 / 8)
        assert ref.close(o, want, bound, torch.bfloat16)
        lens += 1
        now = [n + 1 for n in now]
    assert pool.device_error() == (0, 0)


@pytest.mark.parametrize("batch_rows", [1, 3])
def test_attention_block(paged, batch_rows):
    """A layer's attention over compressed projections, token after token behind a
    prompt taken in one chunk, against 64 bits from the same rounded inputs."""
    from lossless_bf16_weight_nwc_b200 import _lib, synth
    hidden, h, hk, dim, page = 256, 4, 2, 64, 16
    w = [synth.matrix(synth.MatrixSpec("w", r, c, "normal", 0.06, 0), i)
         for i, (r, c) in enumerate([(h * dim, hidden), (hk * dim, hidden), (hk * dim, hidden),
                                     (hidden, h * dim)])]
    wf = [torch.from_numpy(synth.bf16_bits_to_float(x).astype(np.float64)).cuda() for x in w]
    g = gen(40)
    kv = paged.PagedKV(*(randn(g, 24, page, hk, dim).bfloat16() for _ in range(2)))
    qw, kw = weights(g, "bf16", dim), weights(g, "f32", dim).bfloat16()
    freq = paged.rope_frequencies(dim, 5e5, factor=8.0)
    block = paged.AttentionBlock(_lib.CompressedMatrix.compress_fused(w[:3]),
                                 _lib.CompressedMatrix.compress(w[3]), kv, freq, qw, kw)
    table = torch.arange(6 * batch_rows, device="cuda").int().view(batch_rows, 6)
    lens = ints([0] * batch_rows)
    batch = paged.PagedBatch(table, lens)
    kept = [[], []]                                    # exact k and v of every token
    at = 0
    for chunk in (17, 1, 1, 1):
        x = randn(g, batch_rows * chunk, hidden).bfloat16()
        lens += chunk
        y = block.step(x, batch)
        pos = (at + torch.arange(chunk, device="cuda")).repeat(batch_rows)
        q, k, v = ((x.double() @ m.T).unflatten(1, (-1, dim)) for m in wf[:3])
        q = ref.norm_rotate(q, qw, pos, freq, False, 1e-6)[0].unflatten(0, (batch_rows, chunk))
        k = ref.norm_rotate(k, kw, pos, freq, False, 1e-6)[0].unflatten(0, (batch_rows, chunk))
        kept[0].append(k)
        kept[1].append(v.unflatten(0, (batch_rows, chunk)))
        ks, vs = (torch.cat(t, 1).repeat_interleave(h // hk, 2) for t in kept)
        s = torch.einsum("bihd,bjhd->bhij", q, ks) / math.sqrt(dim)
        i = at + torch.arange(chunk, device="cuda")
        s = s.masked_fill(torch.arange(at + chunk, device="cuda") > i[:, None], -math.inf)
        o = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), vs)
        want = o.flatten(2).flatten(0, 1) @ wf[3].T
        # q, k, v, p and o are rounded to BF16 once each: 2^-8 at most, of which a
        # score of size |s| takes 2 |s| 2^-8 into its weight.
        top = float(torch.einsum("bihd,bjhd->bhij", q.abs(), ks.abs()).max() / math.sqrt(dim))
        part = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), vs.abs()).flatten(2).flatten(0, 1)
        bound = (part @ wf[3].abs().T) * 2.0 ** -8 * (3 + 4 * top)
        assert bool(((y.double() - want).abs() <= bound).all())
        rel = float((y.double() - want).norm() / want.norm())
        assert rel <= 2.0 ** -8 * (3 + 4 * top)
        at += chunk
    assert kv.device_error() == (0, 0)


@pytest.mark.parametrize("rows", [1, 20, 61])
def test_attention_block_captured(paged, rows):
    """A captured step replayed token after token gives the eager steps' bits; lengths
    and inputs change in place."""
    from lossless_bf16_weight_nwc_b200 import _lib, synth
    hidden, h, hk, dim = 512, 8, 2, 64
    w = [synth.matrix(synth.MatrixSpec("w", r, c, "normal", 0.06, 0), i)
         for i, (r, c) in enumerate([(h * dim, hidden), (hk * dim, hidden), (hk * dim, hidden),
                                     (hidden, h * dim)])]
    wqkv, wo = _lib.CompressedMatrix.compress_fused(w[:3]), _lib.CompressedMatrix.compress(w[3])
    freq, sides = paged.rope_frequencies(dim), []
    table = torch.randperm(3 * rows, generator=gen(41), device="cuda").int().view(rows, 3)
    for _ in range(2):
        kv = paged.PagedKV(*(torch.zeros(3 * rows, 16, hk, dim, dtype=torch.bfloat16,
                                         device="cuda") for _ in range(2)))
        lens = ints([1 + i % 7 for i in range(rows)])
        sides.append((paged.AttentionBlock(wqkv, wo, kv, freq), paged.PagedBatch(table, lens),
                      lens, kv))
    g = gen(42)
    x = randn(g, rows, hidden).bfloat16()
    block, batch, lens, kv = sides[1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, batch)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, batch)
    for _ in range(30):
        want = sides[0][0].step(x, sides[0][1])
        graph.replay()
        assert torch.equal(y, want) and torch.equal(bits(kv.k_pages), bits(sides[0][3].k_pages))
        x.copy_(randn(g, rows, hidden))
        for s in sides:
            s[2].add_(1)
    assert kv.device_error() == (0, 0) and wqkv.device_error() == (0, 0)
