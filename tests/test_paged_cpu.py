"""The paged operators without a GPU: what the C ABI and the Python calls refuse
before anything is launched, and the frequencies."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

OK, INVALID = 0, 1


@pytest.fixture(scope="module")
def lib():
    from lossless_bf16_weight_nwc_b200 import build
    build.build()
    from lossless_bf16_weight_nwc_b200 import _lib
    return _lib


def heads(lib, type_=1, data=0x10000, ts=2048, hs=128):
    return lib.nwc_heads(ctypes.sizeof(lib.nwc_heads), type_, data, ts, hs)


def rope(lib, **kw):
    r = lib.nwc_rope(ctypes.sizeof(lib.nwc_rope), 128, 0, 0, 0x20000, 0x30000, 0x40000, 1e-6)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def cache(lib, **kw):
    c = lib.nwc_kv_cache(ctypes.sizeof(lib.nwc_kv_cache), 16, 8, 128, 100, 0x100000, 0x200000,
                         16384, 1024, 128, 16384, 1024, 128, 0x5000)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def batch(lib, **kw):
    b = lib.nwc_kv_batch(ctypes.sizeof(lib.nwc_kv_batch), 0, 1, 0x1000, 4, 4, 0x2000, None, 0,
                         None, None, 0, 0, None)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def test_qk_norm_rope_arguments(lib):
    q, out, k, ko = heads(lib), heads(lib, 0), heads(lib), heads(lib, 0)

    def status(**kw):
        a = dict(q=q, k=k, q_out=out, k_out=ko, tokens=0, heads=16, kv_heads=4, dim=128,
                 pos=0x8000, wide=1, rope=rope(lib))
        a.update(kw)
        return lib.LIB.nwc_qk_norm_rope(a["q"], a["k"], a["q_out"], a["k_out"], a["tokens"],
                                        a["heads"], a["kv_heads"], a["dim"], a["pos"], a["wide"],
                                        a["rope"], None)

    assert status() == OK                              # no tokens: nothing to launch
    assert status(q=None, q_out=None) == OK and status(k=None, k_out=None, kv_heads=0) == OK
    bad = [dict(q=None), dict(k_out=None), dict(q=None, q_out=None, k=None, k_out=None),
           dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(heads=0), dict(kv_heads=0),
           dict(dim=0), dict(dim=12), dict(dim=264), dict(pos=None), dict(pos=0x8004),
           dict(rope=None), dict(k=heads(lib, 0)), dict(k_out=heads(lib, 1)),
           dict(q=heads(lib, 2)), dict(q=heads(lib, data=None)), dict(q=heads(lib, data=0x10002)),
           dict(q=heads(lib, ts=-1)), dict(q=heads(lib, hs=1 << 40)),
           dict(rope=rope(lib, rotary_dim=136)), dict(rope=rope(lib, rotary_dim=12)),
           dict(rope=rope(lib, rotary_dim=-8)), dict(rope=rope(lib, d_freq=None)),
           dict(rope=rope(lib, d_freq=0x20004)), dict(rope=rope(lib, eps=-1.0)),
           dict(rope=rope(lib, eps=math.nan)), dict(rope=rope(lib, eps=math.inf)),
           dict(rope=rope(lib, weight_type=2)), dict(rope=rope(lib, d_k_weight=0x40001)),
           dict(rope=rope(lib, struct_size=8))]
    for kw in bad:
        assert status(**kw) == INVALID, kw
    assert status(rope=rope(lib, rotary_dim=0, d_freq=None)) == OK


CACHE_BAD = [dict(page_size=12), dict(page_size=4), dict(page_size=1 << 21), dict(kv_heads=0),
             dict(dim=12), dict(dim=264), dict(pages=0), dict(pages=1 << 31), dict(d_k=None),
             dict(d_v=0x200008), dict(k_token_stride=1028), dict(v_head_stride=-8),
             dict(k_page_stride=1 << 40), dict(d_error=None), dict(d_error=0x5002),
             dict(struct_size=0)]
BATCH_BAD = [dict(sequences=-1), dict(new_tokens=0), dict(sequences=1 << 20, new_tokens=1 << 10),
             dict(groups=-1), dict(groups=1), dict(struct_size=4),
             dict(sequences=2, table_width=-1), dict(sequences=2, d_block_table=None),
             dict(sequences=2, d_seq_lens=None), dict(sequences=2, d_seq_lens=0x2002),
             dict(sequences=2, table_stride=-1), dict(sequences=2, d_q_lens=0x2001),
             dict(sequences=2, groups=1, prefix_width=1, d_prefix_table=0x100, d_prefix_lens=0x100),
             dict(sequences=2, groups=1, prefix_width=-1, d_prefix_table=0x100, d_prefix_lens=0x100,
                  d_group_start=0x100),
             dict(sequences=2, groups=1, prefix_width=1, d_prefix_lens=0x100, d_group_start=0x100)]


def test_append_arguments(lib):
    k, v, q, qo = heads(lib), heads(lib), heads(lib), heads(lib, 0)

    def status(c=None, b=None, **kw):
        a = dict(q=q, q_out=qo, heads=16, k=k, v=v, rope=rope(lib))
        a.update(kw)
        return lib.LIB.nwc_kv_append(c or cache(lib), b or batch(lib), a["q"], a["q_out"],
                                     a["heads"], a["k"], a["v"], a["rope"], None)

    assert status() == OK and status(q=None, q_out=None, heads=0) == OK
    for kw in CACHE_BAD:
        assert status(c=cache(lib, **kw)) == INVALID, kw
    for kw in BATCH_BAD:
        assert status(b=batch(lib, **kw)) == INVALID, kw
    for kw in (dict(q=None), dict(q_out=None), dict(k=None), dict(v=None), dict(v=heads(lib, 0)),
               dict(q=heads(lib, 0)), dict(q_out=heads(lib, 1)), dict(heads=0), dict(rope=None),
               dict(rope=rope(lib, rotary_dim=136))):
        assert status(**kw) == INVALID, kw


def test_attention_arguments(lib):
    q, out = heads(lib, 0), heads(lib, 0)

    def status(c=None, b=None, **kw):
        a = dict(q=q, heads=16, scale=0.1, out=out, lse=None, ws=0x10000, bytes=1 << 40)
        a.update(kw)
        return lib.LIB.nwc_kv_attention(c or cache(lib), b or batch(lib), a["q"], a["heads"],
                                        a["scale"], a["out"], a["lse"], a["ws"], a["bytes"], None)

    for kw in CACHE_BAD:
        assert status(c=cache(lib, **kw)) == INVALID, kw
    for kw in BATCH_BAD:
        assert status(b=batch(lib, **kw)) == INVALID, kw
    for kw in (dict(q=None), dict(out=None), dict(q=heads(lib, 1)), dict(out=heads(lib, 1)),
               dict(q=heads(lib, 0, data=0x10008)), dict(out=heads(lib, 0, ts=2052)),
               dict(heads=0), dict(heads=12), dict(scale=math.nan), dict(scale=math.inf),
               dict(lse=2)):
        assert status(**kw) == INVALID, kw
    assert status(c=cache(lib, kv_heads=1), b=batch(lib, sequences=1 << 20), heads=2048) == INVALID
    for dim in (8, 96, 256):
        assert status(c=cache(lib, dim=dim)) == 2      # NWC_ERR_UNSUPPORTED
    n = ctypes.c_uint64()
    ask = lib.LIB.nwc_kv_attention_workspace
    assert ask(cache(lib), batch(lib), 12, ctypes.byref(n)) == INVALID
    assert ask(cache(lib), batch(lib), 16, None) == INVALID
    assert ask(cache(lib, dim=96), batch(lib), 16, ctypes.byref(n)) == 2
    assert lib.LIB.nwc_kv_get_error(None, None, None) == INVALID


def test_attention_scales(lib):
    """Refused where the kernel's own unit, scale / ln 2, would be infinite."""
    q, out = heads(lib, 0), heads(lib, 0)
    for scale, want in ((2e38, OK), (-2e38, OK), (0.0, OK), (2.4e38, INVALID), (-3e38, INVALID)):
        got = lib.LIB.nwc_kv_attention(cache(lib), batch(lib), q, 16, scale, out, None, 0x10000,
                                       1 << 40, None)
        assert got == want, scale


def test_python_calls_refuse_host_tensors_and_gradients(lib):
    from lossless_bf16_weight_nwc_b200 import paged
    q = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        paged.qk_norm_rope(q, q, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        paged.qk_norm_rope(None, [1.0], None)
    with pytest.raises(ValueError, match="CUDA"):
        paged.PagedKV(torch.zeros(4, 16, 2, 64), torch.zeros(4, 16, 2, 64))
    with pytest.raises(ValueError, match="CUDA"):
        paged.PagedBatch(torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="gradient"):
        paged._no_grad(None, torch.zeros(1, requires_grad=True))
    with torch.no_grad():
        paged._no_grad(torch.zeros(1, requires_grad=True))


def test_tensor_checks(lib):
    """The checks behind every call, on host tensors."""
    from lossless_bf16_weight_nwc_b200 import paged
    cpu = torch.device("cpu")
    t = torch.zeros(3, 4, 64)

    def view(*args, **kw):
        return lib.nwc_heads.from_buffer_copy(paged._heads(*args, **kw))

    v = view(t, "t", (3, 4, 64), cpu)
    assert (v.struct_size, v.type, v.d_data) == (ctypes.sizeof(v), 1, t.data_ptr())
    assert (v.token_stride, v.head_stride) == (256, 64)
    assert view(t[:1], "t", (1, 4, 64), cpu).token_stride == 0
    with pytest.raises(TypeError):
        paged._heads(t.half(), "t", (3, 4, 64), cpu)
    with pytest.raises(ValueError, match="shape"):
        paged._heads(t, "t", (3, 4, 32), cpu)
    with pytest.raises(ValueError, match="contiguous"):
        paged._heads(t.transpose(1, 2), "t", (3, 64, 4), cpu)
    with pytest.raises(ValueError, match="expected cuda"):
        paged._heads(t, "t", (3, 4, 64), torch.device("cuda:0"))
    paged._heads(t.transpose(0, 1), "o", (4, 3, 64), cpu, output=True)
    paged._heads(t[..., 8:], "o", (3, 4, 56), cpu, wide=True)
    for bad in (t[..., 1:57], torch.as_strided(t, (3, 4, 56), (256, 60, 1))):
        with pytest.raises(ValueError, match="alignment"):
            paged._heads(bad, "o", (3, 4, 56), cpu, wide=True)
    for bad in (t[:, :1].expand(3, 4, 64), t[:1].expand(3, 4, 64),
                torch.as_strided(t, (3, 4, 64), (64, 64, 1))):
        with pytest.raises(ValueError, match="overlap"):
            paged._heads(bad, "o", (3, 4, 64), cpu, output=True)
    f = torch.ones(32, dtype=torch.float64)
    k = torch.ones(64)
    r = lib.nwc_rope.from_buffer_copy(paged._rope(64, cpu, f, None, k, 1e-6, True))
    assert (r.struct_size, r.rotary_dim, r.interleaved, r.weight_type) == (
        ctypes.sizeof(r), 64, 1, 1)
    assert (r.d_freq, r.d_q_weight, r.d_k_weight) == (f.data_ptr(), None, k.data_ptr())
    assert math.isclose(r.eps, 1e-6, rel_tol=1e-6)
    for bad in (f[:30], torch.ones(64, dtype=torch.float64), f.float(), f[::2], [1.0]):
        with pytest.raises((ValueError, TypeError)):
            paged._rope(64, cpu, bad, None, None, 1e-6, False)
    with pytest.raises(TypeError, match="one dtype"):
        paged._rope(64, cpu, f, torch.ones(64).bfloat16(), torch.ones(64), 1e-6, False)
    with pytest.raises(ValueError, match="eps"):
        paged._rope(64, cpu, f, None, None, -1.0, False)


def test_outputs_with_gaps(lib):
    """Every layout without two elements at one place is an output: the last head or
    token need not bring its gap with it."""
    from lossless_bf16_weight_nwc_b200 import paged
    cpu = torch.device("cpu")
    t = torch.zeros(3, 5, 64)
    for out in (t[:, ::2], t[..., 8:], t.transpose(0, 1)[:, ::2], t[::2].transpose(0, 1),
                torch.as_strided(t, (2, 2, 8), (24, 16, 1)),
                torch.as_strided(t, (2, 2, 8), (16, 24, 1))):
        paged._heads(out, "o", out.shape, cpu, output=True)
    for strides in ((23, 16, 1), (16, 23, 1), (7, 24, 1), (24, 7, 1)):
        bad = torch.as_strided(t, (2, 2, 8), strides)
        with pytest.raises(ValueError, match="overlap"):
            paged._heads(bad, "o", bad.shape, cpu, output=True)


def test_package_names(lib):
    import lossless_bf16_weight_nwc_b200 as package
    from lossless_bf16_weight_nwc_b200 import paged
    for name in ("AttentionBlock", "PagedBatch", "PagedKV", "qk_norm_rope", "rope_frequencies"):
        assert name in package.__all__ and getattr(package, name) is getattr(paged, name)
    assert all(hasattr(package, name) for name in package.__all__)
    with pytest.raises(AttributeError):
        package.no_such_name


def test_tangents_are_refused(lib):
    """Forward-mode gradients, which torch.no_grad() leaves on."""
    import torch.autograd.forward_ad as fwd
    from lossless_bf16_weight_nwc_b200 import paged
    plain = torch.ones(3)
    with fwd.dual_level():
        dual = fwd.make_dual(plain, torch.ones(3))
        paged._no_grad(None, plain, [1], fwd.unpack_dual(dual).primal)
        with pytest.raises(ValueError, match="tangent"):
            paged._no_grad(None, plain, dual)
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
            paged._no_grad(dual)
    paged._no_grad(plain)


def test_attention_block_arguments(lib):
    """What a step would find out after it has appended is refused when the block is made."""
    from types import SimpleNamespace as Fake
    from lossless_bf16_weight_nwc_b200 import paged
    cpu = torch.device("cpu")

    def block(heads=8, kv_heads=2, dim=64, cols=None, wqkv_on=cpu, wo_on=cpu, splits=None, **kw):
        b = splits or [0, heads * dim, (heads + kv_heads) * dim, (heads + 2 * kv_heads) * dim]
        return paged.AttentionBlock(
            Fake(row_splits=b, image=Fake(device=wqkv_on)),
            Fake(cols=heads * dim if cols is None else cols, image=Fake(device=wo_on)),
            Fake(kv_heads=kv_heads, dim=dim, device=cpu),
            kw.pop("freq", torch.ones(dim // 2, dtype=torch.float64)), **kw)

    block(), block(dim=128, scale=-1.0), block(kv_heads=1, heads=3, q_weight=torch.ones(64))
    other = torch.device("cuda:0")
    for bad in (dict(heads=7), dict(heads=0), dict(dim=32), dict(dim=80), dict(cols=64),
                dict(scale=math.inf), dict(scale=math.nan), dict(scale=3e38), dict(eps=-1.0),
                dict(wqkv_on=other), dict(wo_on=other), dict(splits=[0, 512]),
                dict(freq=torch.ones(30, dtype=torch.float64)), dict(q_weight=torch.ones(32)),
                dict(k_weight=torch.ones(64, device="meta"))):
        with pytest.raises(ValueError):
            block(**bad)


def _bytes_of(t):
    """Every byte of a tensor, one by one."""
    at = [t.data_ptr()]
    for n, s in zip(t.shape, t.stride()):
        at = [a + i * s * t.element_size() for a in at for i in range(n)]
    return {a + b for a in at for b in range(t.element_size())}


def test_outputs_apart(lib):
    """Two views of one memory, told apart byte by byte; the output itself as source."""
    import random
    from lossless_bf16_weight_nwc_b200 import paged
    rng = random.Random(3)
    base = torch.zeros(400, dtype=torch.bfloat16)
    apart = met = 0
    for _ in range(3000):
        strides = rng.choice([(24, 8), (8, 24), (40, 10), (16, 16), (30, 0), (7, 3), (0, 0)])
        a, b = (torch.as_strided(base, (rng.randint(1, 4), rng.randint(1, 3), rng.randint(1, 9)),
                                 (*strides, 1), rng.randint(0, 150)) for _ in range(2))
        both = not _bytes_of(a).isdisjoint(_bytes_of(b))
        assert paged._meet(a, b) == both and paged._meet(b, a) == both
        met, apart = met + both, apart + (not both)
    assert min(met, apart) > 500
    y = torch.zeros(5, 6 * 8).bfloat16()
    q, k = y[:, :32].unflatten(1, (4, 8)), y[:, 32:].unflatten(1, (2, 8))
    paged._apart(q, "o", q, k, None, torch.zeros(3))
    paged._apart(k, "o", q, torch.zeros(0))
    paged._apart(q[:1], "o", q[:1], k)                     # strides of one token do not count
    paged._apart(torch.zeros(0, 4, 8).bfloat16(), "o", q)
    paged._apart(torch.zeros(5, 4, 8), "o", q)
    full = torch.zeros(10, 4, 8)
    for out, source, others in (
            (k, k, (q, y)), (q[1:], q[:-1], ()), (full[:5].bfloat16(), None, ()),
            (torch.as_strided(full.view(torch.bfloat16), (5, 4, 8), (64, 16, 1)), full[:5], ()),
            (torch.as_strided(full, (5, 4, 8), (32, 8, 1)), full[:5].transpose(0, 1), ()),
            (full[:5], None, (full[4, 3],)), (q, q, (y[:, 31:40],)), (q, q, (q,))):
        if others or source is not None:
            with pytest.raises(ValueError, match="overlaps"):
                paged._apart(out, "o", source, *others)


def test_rope_frequencies(lib):
    from lossless_bf16_weight_nwc_b200 import paged
    f = paged.rope_frequencies(128, 5e5, "cpu")
    assert f.dtype == torch.float64 and f.shape == (64,) and f[0] == 1
    assert math.isclose(float(f[63]), 5e5 ** (-126 / 128), rel_tol=1e-14)
    g = paged.rope_frequencies(128, 5e5, "cpu", factor=8.0)
    turns = 8192 * f / (2 * math.pi)
    assert torch.equal(g[turns > 4], f[turns > 4])
    assert torch.allclose(g[turns < 1], f[turns < 1] / 8, rtol=1e-14, atol=0)
    middle = (turns >= 1) & (turns <= 4)
    assert middle.any() and (g[middle] <= f[middle]).all() and (g[middle] >= f[middle] / 8).all()
    for bad in (0, 7):
        with pytest.raises(ValueError):
            paged.rope_frequencies(bad, device="cpu")
